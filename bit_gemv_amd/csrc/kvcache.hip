// kvcache.hip -- quantizing keys and values into the paged cache as they are
// written (kv_cache_write) and reading them back (kv_cache_read).
//
// A team of D / 8 lanes takes one head of four neighbouring tokens (an aligned
// quad of positions, the unit in which the cache stores values), 8 elements a
// lane: statistics by a butterfly over the team, then codes. Keys leave as
// one run of bytes per token and lane, values as whole words of four tokens
// (single bytes where only some of the quad's tokens are new). Both kernels
// are bound by HBM on chunks (21k tokens, 8 heads of 128, INT8: writing 31.6 us,
// 4.2 TB/s; reading 25 us, 5.3) and by latency on a decode batch (4.8 and 3.6).
#include "common.hpp"
#include "kv.hpp"

namespace lq {

namespace {

constexpr int kTpb = 256;

// 8 elements as they lie, and as fp32
template <bool F32>
struct Raw {
    u32x4 a[F32 ? 2 : 1];
};
template <bool F32>
LQ_DEVICE Raw<F32> load_row8(const void *p, int64_t e) {
    Raw<F32> r;
    const u32x4 *q = reinterpret_cast<const u32x4 *>(static_cast<const char *>(p) + e * (F32 ? 4 : 2));
    r.a[0] = q[0];
    if constexpr (F32) r.a[1] = q[1];
    return r;
}
template <bool F32>
LQ_DEVICE void widen_row8(const Raw<F32> &r, bool in, float *f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = F32 ? r.a[F32 ? j / 4 : 0][j % 4] : r.a[0][j / 2];
        const float v = F32 ? __uint_as_float(w) : j % 2 ? bf16_hi(w) : bf16_lo(w);
        f[j] = in ? v : 0.0f;
    }
}

// Maximum over the team's W (8, 16 or 32) lanes.
template <int W>
LQ_DEVICE float lanes_max(float v) {
    v = fmaxf(v, dpp_f32<kDppXor1>(v));
    v = fmaxf(v, dpp_f32<kDppXor2>(v));
    v = fmaxf(v, dpp_f32<kDppHalfMirror>(v));
    if constexpr (W >= 16) v = fmaxf(v, dpp_f32<kDppMirror>(v));
    if constexpr (W >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

// Scale, zero and codes (stored unsigned) of the team's D elements, 8 in this
// lane: quantize_groupwise's formulas, except that the scale is the range
// times the fp32 reciprocal of the level count, at most one ulp from the
// quotient. That is how torch divides a GPU tensor by a number, so the cache
// holds what the formulas written in torch give, bit for bit; the quotient
// (no slower through div_rn) puts a code or a zero one off from theirs where
// its rounding lies within that ulp. The code is in the low byte of c.
// Quotients x / s go through div_rn (common.hpp) while every magnitude is at
// most 2^59: s is then in [1e-8 / 256, 2^60], so that a quotient of 1/2 or more
// has |x| >= s / 2 and every intermediate is normal; smaller ones round to 0
// either way. (The IEEE division sequence took the kernel from HBM's rate to
// the instruction rate: 45 us for 21k tokens of the 70B heads.)
template <int BITS, bool SYM, bool FAST>
LQ_DEVICE void codes8(const float *x, float s, float z, uint32_t *c) {
    const float y = 1.0f / s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float q = FAST ? div_rn(x[j], s, y) : x[j] / s;
        if constexpr (SYM) {
            constexpr float mid = (float)(1 << (BITS - 1));
            // |q| <= (mid - 1)(1 + 2^-21), so no clamp is needed; floats from
            // 2^23 are integers, so the sum rounds q (ties to even) and holds
            // q + mid in its low byte
            c[j] = __float_as_uint(q + (8388608.0f + mid));
        } else {
            c[j] = (uint32_t)(int)clamp_code(rintf(q) + z, 0.0f, (float)((1 << BITS) - 1));
        }
    }
}

template <int D, int BITS, bool SYM>
LQ_DEVICE void encode8(const float *x, float &s, float &z, uint32_t *c) {
    constexpr int W = D / 8;
    float top;  // largest magnitude
    if constexpr (SYM) {
        constexpr float qmax = (float)((1 << (BITS - 1)) - 1);
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(x[j]));
        top = lanes_max<W>(a);
        s = (top < kFloor ? kFloor : top) * (1.0f / qmax);
        z = 0.0f;
    } else {
        constexpr float levels = (float)((1 << BITS) - 1);
        float lo = x[0], hi = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            lo = fminf(lo, x[j]);
            hi = fmaxf(hi, x[j]);
        }
        lo = -lanes_max<W>(-lo);
        hi = lanes_max<W>(hi);
        const float range = hi - lo;
        s = (range < kFloor ? kFloor : range) * (1.0f / levels);
        z = rintf(-lo / s) + 0.0f;  // -0 -> +0
        top = fmaxf(fabsf(lo), fabsf(hi));
    }
    if (__all(top <= 5.76460752303423488e+17f))  // 2^59
        codes8<BITS, SYM, true>(x, s, z, c);
    else
        codes8<BITS, SYM, false>(x, s, z, c);
}

// four low bytes to a word
LQ_DEVICE uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u),
                                 0x05040100u);
}

// A sequence's items: aligned quads of its rows' positions (READ: those below
// zero as well), for each two sides of every head.
struct Items {
    int64_t quad0, count;
};
template <bool READ>
LQ_DEVICE Items items_of(const KvRows &rows, int heads) {
    if (rows.n == 0 || (!READ && rows.first + rows.n <= 0)) return {0, 0};
    const int64_t quad0 = (!READ && rows.first < 0 ? 0 : rows.first) >> 2;
    return {quad0, (((rows.first + rows.n - 1) >> 2) - quad0 + 1) * 2 * heads};
}

// Where a team starts and how it goes on. In the plain grid blocks in x are a
// sequence's items and blocks in y the sequences. In the flat one block
// blockIdx.x is that block of all sequences' blocks of items, one after
// another: each wave adds the sequences up, 64 at a time.
struct Walk {
    int64_t seq, seq_step, item, item_step;
};
template <bool READ>
LQ_DEVICE Walk walk_of(const KvBatch &bt, int shift, int heads, int flat, int teams, int team) {
    if (!flat) return {blockIdx.y, gridDim.y, (int64_t)blockIdx.x * teams + team, (int64_t)gridDim.x * teams};
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int64_t s0 = 0; s0 < bt.b; s0 += 64) {
        int64_t mine = 0;
        if (s0 + lane < bt.b)
            mine = (items_of<READ>(kv_rows(bt, s0 + lane, shift), heads).count + teams - 1) / (uint32_t)teams;
        const int64_t upto = before + scan64(mine);
        const uint64_t past = __ballot(upto > (int64_t)blockIdx.x);
        if (past) {
            const int src = __ffsll((unsigned long long)past) - 1;
            const int64_t first = readlane64(upto - mine, src);
            return {s0 + src, (int64_t)1 << 60, (blockIdx.x - first) * teams + team, (int64_t)1 << 60};
        }
        before = readlane64(upto, 63);
    }
    return {bt.b, 1, 0, 1};
}

// which sequence, quad of positions, head and side (key or value) a team has
struct Item {
    int64_t quad;
    int head, side;
};

template <int D>
LQ_DEVICE Item item_of(int64_t i, int heads, int64_t quad0) {
    Item it;
    int64_t j;
    if (i >> 32) {
        j = i / heads;
    } else {
        j = (uint32_t)i / (uint32_t)heads;
    }
    it.head = (int)(i - j * heads);
    it.side = (int)(j & 1);
    it.quad = quad0 + (j >> 1);
    return it;
}

template <int D, int BITS, bool SYM, bool F32>
__global__ __launch_bounds__(kTpb) void kv_write_kernel(KvWriteArgs a) {
    constexpr int W = D / 8;                 // lanes of a team
    constexpr int kRow = D * BITS / 8;       // bytes of a token's codes
    constexpr int kLane = BITS;              // of them, this lane's 8 elements
    const int lane = threadIdx.x % W, team = threadIdx.x / W;
    const Walk w0 = walk_of<false>(a.batch, a.c.page_shift, a.c.heads, a.flat, kTpb / W, team);
    for (int64_t seq = w0.seq; seq < a.batch.b; seq += w0.seq_step) {
        const KvRows rows = kv_rows(a.batch, seq, a.c.page_shift);
        const Items mine = items_of<false>(rows, a.c.heads);
        const int64_t quad0 = mine.quad0;
        for (int64_t i = w0.item; i < mine.count; i += w0.item_step) {
            const Item it = item_of<D>(i, a.c.heads, quad0);
            const int64_t page = kv_page(a.batch, seq, it.quad * 4, a.c.page_shift, a.c.pages);
            if (page < 0) continue;
            const void *src = it.side ? a.v : a.k;
            const int64_t stride = it.side ? a.v_stride : a.k_stride;
            uint32_t code[4][8];
            float s[4], z[4];
            bool in[4];
            // all four rows' loads at once: rows that are not the call's read a
            // neighbour instead
            Raw<F32> raw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                int64_t row = it.quad * 4 + u - rows.first;
                in[u] = row >= 0 && row < rows.n;
                row = row < 0 ? 0 : row < rows.n ? row : rows.n - 1;
                raw[u] = load_row8<F32>(src, (rows.begin + row) * stride + (int64_t)it.head * D + lane * 8);
            }
            float x[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) widen_row8<F32>(raw[u], in[u], x[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) encode8<D, BITS, SYM>(x[u], s[u], z[u], code[u]);
            const int64_t slot = ((page * a.c.heads + it.head) << a.c.page_shift) +
                                 ((it.quad * 4) & ((1 << a.c.page_shift) - 1));
            // bytes of this lane: 8 (bits 8) or 4 (bits 4) per token
            if (BITS == 4) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) code[u][j] = (code[u][2 * j] & 15u) | (code[u][2 * j + 1] << 4);
            }
            float *scales = it.side ? a.c.v_scales : a.c.k_scales;
            float *zeros = it.side ? a.c.v_zeros : a.c.k_zeros;
            if (lane == 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (in[u]) {
                        scales[slot + u] = s[u];
                        if (!SYM) zeros[slot + u] = z[u];
                    }
            }
            if (it.side == 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (!in[u]) continue;
                    uint32_t w[kLane / 4];
#pragma unroll
                    for (int j = 0; j < kLane / 4; ++j)
                        w[j] = pack_bytes(code[u][4 * j], code[u][4 * j + 1], code[u][4 * j + 2], code[u][4 * j + 3]);
                    uint32_t *p = reinterpret_cast<uint32_t *>(a.c.k_codes + (slot + u) * kRow + lane * kLane);
#pragma unroll
                    for (int j = 0; j < kLane / 4; ++j) p[j] = w[j];
                }
            } else {
                uint8_t *p = a.c.v_codes + slot * kRow + (int64_t)lane * kLane * 4;
                if (in[0] && in[1] && in[2] && in[3]) {
                    u32x4 w[kLane / 4];
#pragma unroll
                    for (int j = 0; j < kLane; ++j)
                        w[j / 4][j % 4] = pack_bytes(code[0][j], code[1][j], code[2][j], code[3][j]);
#pragma unroll
                    for (int j = 0; j < kLane / 4; ++j) reinterpret_cast<u32x4 *>(p)[j] = w[j];
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (in[u])
#pragma unroll
                            for (int j = 0; j < kLane; ++j) p[j * 4 + u] = (uint8_t)code[u][j];
                }
            }
        }
    }
}

template <int D, int BITS, bool SYM, bool F32>
__global__ __launch_bounds__(kTpb) void kv_read_kernel(KvReadArgs a) {
    constexpr int W = D / 8;
    constexpr int kRow = D * BITS / 8;
    constexpr int kLane = BITS;
    const int lane = threadIdx.x % W, team = threadIdx.x / W;
    const Walk w0 = walk_of<true>(a.batch, a.c.page_shift, a.c.heads, a.flat, kTpb / W, team);
    for (int64_t seq = w0.seq; seq < a.batch.b; seq += w0.seq_step) {
        const KvRows rows = kv_rows(a.batch, seq, a.c.page_shift);
        const Items mine = items_of<true>(rows, a.c.heads);
        const int64_t quad0 = mine.quad0;
        for (int64_t i = w0.item; i < mine.count; i += w0.item_step) {
            const Item it = item_of<D>(i, a.c.heads, quad0);
            void *dst = it.side ? a.v : a.k;
            if (!dst) continue;
            const int64_t page = kv_page(a.batch, seq, it.quad * 4, a.c.page_shift, a.c.pages);
            const int64_t slot = page < 0 ? 0
                                          : ((page * a.c.heads + it.head) << a.c.page_shift) +
                                                ((it.quad * 4) & ((1 << a.c.page_shift) - 1));
            const float *scales = it.side ? a.c.v_scales : a.c.k_scales;
            const float *zeros = it.side ? a.c.v_zeros : a.c.k_zeros;
            uint32_t w[4][kLane / 4];  // this lane's code bytes of each token
            float s[4], z[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s[u] = 0.0f;
                z[u] = SYM ? (float)(1 << (BITS - 1)) : 0.0f;
#pragma unroll
                for (int j = 0; j < kLane / 4; ++j) w[u][j] = 0;
            }
            if (page >= 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    s[u] = scales[slot + u];
                    if (!SYM) z[u] = zeros[slot + u];
                }
                if (it.side == 0) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t *p =
                            reinterpret_cast<const uint32_t *>(a.c.k_codes + (slot + u) * kRow + lane * kLane);
#pragma unroll
                        for (int j = 0; j < kLane / 4; ++j) w[u][j] = p[j];
                    }
                } else {
                    const u32x4 *p =
                        reinterpret_cast<const u32x4 *>(a.c.v_codes + slot * kRow + (int64_t)lane * kLane * 4);
#pragma unroll
                    for (int j = 0; j < kLane / 4; ++j) {
                        const u32x4 q = p[j];  // four elements' words of four tokens
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            w[u][j] = ((q[0] >> (8 * u)) & 255u) | (((q[1] >> (8 * u)) & 255u) << 8) |
                                      (((q[2] >> (8 * u)) & 255u) << 16) | (((q[3] >> (8 * u)) & 255u) << 24);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t row = it.quad * 4 + u - rows.first;
                if (row < 0 || row >= rows.n) continue;
                const bool live = page >= 0 && it.quad * 4 + u >= 0;
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t c = BITS == 8 ? (w[u][j / 4] >> (8 * (j % 4))) & 255u : (w[u][0] >> (4 * j)) & 15u;
                    f[j] = live ? ((float)c - z[u]) * s[u] : 0.0f;
                }
                const int64_t e = ((rows.begin + row) * a.c.heads + it.head) * D + lane * 8;
                if constexpr (F32) {
                    f32x4 *p = reinterpret_cast<f32x4 *>(static_cast<float *>(dst) + e);
                    p[0] = f32x4{f[0], f[1], f[2], f[3]};
                    p[1] = f32x4{f[4], f[5], f[6], f[7]};
                } else {
                    u32x4 v;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bf16x2_t b{(__bf16)f[2 * j], (__bf16)f[2 * j + 1]};
                        v[j] = __builtin_bit_cast(uint32_t, b);
                    }
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(dst) + e) = v;
                }
            }
        }
    }
}

// The plain grid covers max_rows rows of every sequence. Where that is many
// times the rows there are (one long chunk among single tokens, or no bound
// given), the flat grid covers the rows. Measured (8 heads of 128, INT8, write):
// 256 single tokens beside a chunk of 8192, plain 293 us, flat 22; 4 beside one
// of 2048 (5 times the rows), plain 6.8, flat 6.1; eight chunks of 1024, plain
// 12.0, flat 13.0; 64 single tokens, plain 4.4, flat 4.9. The plain grid walks on
// past its limits.
dim3 kv_grid(const KvCache &c, const KvBatch &bt, int64_t max_rows, int *flat) {
    const int64_t n = max_rows <= 0 || max_rows > bt.rows ? bt.rows : max_rows;
    const int64_t teams = kTpb / (c.head_dim / 8);
    auto blocks = [&](int64_t quads) { return (quads * 2 * c.heads + teams - 1) / teams; };
    int64_t x = blocks((n + 2) / 4 + 1);
    // at most: a quad more at each end of a sequence's rows, a block not full
    const int64_t all = blocks(bt.rows / 4 + 2 * bt.b) + bt.b;
    *flat = x * bt.b > 4 * all && all <= (1 << 23);
    if (*flat) return dim3((uint32_t)all);
    if (x > 65536) x = 65536;
    return dim3((uint32_t)x, (uint32_t)(bt.b < 32768 ? bt.b : 32768));
}

}  // namespace

#define LQ_KV(D, BITS, SYM, F32) \
    if (a.c.head_dim == D && a.c.bits == BITS && (a.c.symmetric != 0) == SYM && (a.f32 != 0) == F32) LQ_KV_DO(D, BITS, SYM, F32)
#define LQ_KV_TYPES(D, BITS, SYM) LQ_KV(D, BITS, SYM, false) LQ_KV(D, BITS, SYM, true)
#define LQ_KV_FORMATS(D) \
    LQ_KV_TYPES(D, 4, false) LQ_KV_TYPES(D, 4, true) LQ_KV_TYPES(D, 8, false) LQ_KV_TYPES(D, 8, true)
#define LQ_KV_ALL LQ_KV_FORMATS(64) LQ_KV_FORMATS(128) LQ_KV_FORMATS(256)

hipError_t launch_kv_write(const KvWriteArgs &args, hipStream_t st) {
    KvWriteArgs a = args;
    const dim3 grid = kv_grid(a.c, a.batch, a.max_rows, &a.flat);
#define LQ_KV_DO(D, BITS, SYM, F32)                                                                        \
    {                                                                                                      \
        hipLaunchKernelGGL((kv_write_kernel<D, BITS, SYM, F32>), grid, dim3(kTpb), 0, st, a);               \
        return hipGetLastError();                                                                          \
    }
    LQ_KV_ALL
#undef LQ_KV_DO
    return hipErrorInvalidValue;
}

hipError_t launch_kv_read(const KvReadArgs &args, hipStream_t st) {
    KvReadArgs a = args;
    const dim3 grid = kv_grid(a.c, a.batch, a.max_rows, &a.flat);
#define LQ_KV_DO(D, BITS, SYM, F32)                                                                        \
    {                                                                                                      \
        hipLaunchKernelGGL((kv_read_kernel<D, BITS, SYM, F32>), grid, dim3(kTpb), 0, st, a);                \
        return hipGetLastError();                                                                          \
    }
    LQ_KV_ALL
#undef LQ_KV_DO
    return hipErrorInvalidValue;
}

}  // namespace lq
