// weigh.hip -- the attention weight that cached tokens receive, summed over a
// call's rows and the heads of a group (kv_cache_weigh).
//
// With codes c, scale s and zero z of a key and a row's log-sum-exp L,
//   weight_j += sum_i exp(scale s_j (q_i . c_j - z_j sum(q_i)) - L_i)
// Products are formed rows x keys: a lane then holds four rows of one key, sums
// them in its own register, and only the last sum crosses lanes. A key belongs
// to one block, which goes through all rows that see it: no workspace, no
// atomics, sums in a fixed order. Keys are bound by HBM for single tokens and by
// the exponentials for chunks: a product of 128 elements is 16 cycles of the
// matrix unit for 64 scores, their exponentials 16 and their scaling and sum 8
// of the vector unit.
#include "codes.hpp"
#include "kv.hpp"

namespace lq {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;

// Steps of STEP keys of all sequences that have rows, one after another; a lane
// a sequence, 64 at a time, the first 64 kept.
struct Place {
    int64_t seq, start;  // start: the sequence's first step among all
    int steps;           // of the sequence
    KvRows rows;
};
template <int STEP>
struct Steps {
    struct Lane {
        KvRows rows;
        int64_t steps, upto;
    };
    const KvBatch &bt;
    const int shift, lane;
    Lane first;

    LQ_DEVICE Lane load(int64_t seq, int64_t before) const {
        Lane x{};
        if (seq < bt.b) {
            x.rows = kv_rows(bt, seq, shift);
            x.steps = x.rows.n > 0 && x.rows.len > 0 ? (x.rows.len + STEP - 1) / STEP : 0;
        }
        x.upto = before + scan64(x.steps);
        return x;
    }
    LQ_DEVICE Steps(const KvBatch &b, int sh, int l) : bt(b), shift(sh), lane(l) { first = load(l, 0); }
    LQ_DEVICE int64_t total() const {
        int64_t sum = readlane64(first.upto, 63);
        for (int64_t s0 = 64; s0 < bt.b; s0 += 64) sum = readlane64(load(s0 + lane, sum).upto, 63);
        return sum;
    }
    // the sequence that holds step pos (below the total)
    LQ_DEVICE Place at(int64_t pos) const {
        Lane x = first;
        for (int64_t s0 = 0;;) {
            const uint64_t past = __ballot(x.upto > pos);
            if (past) {
                const int src = __ffsll((unsigned long long)past) - 1;
                Place p;
                p.seq = s0 + src;
                p.steps = (int)readlane64(x.steps, src);
                p.start = readlane64(x.upto, src) - p.steps;
                p.rows = {readlane64(x.rows.begin, src), readlane64(x.rows.n, src), readlane64(x.rows.first, src),
                          readlane64(x.rows.len, src)};
                return p;
            }
            const int64_t before = readlane64(x.upto, 63);
            s0 += 64;
            if (s0 >= bt.b) return Place{0, pos, 1, KvRows{0, 0, 0, 0}};  // not reached: pos is below the total
            x = load(s0 + lane, before);
        }
    }
};

// ---- few rows: keys streamed past one tile of 16 rows ----
//
// Wave w of a block walks its span's 32-key tiles w, w + 4, ...; the next
// tile's codes are asked for as soon as this one's have been multiplied.
template <int D, int BITS>
struct Few {
    static constexpr int kRow = D * BITS / 8;    // code bytes of a key
    static constexpr int KW = D * BITS / 128;    // code words per lane of 16 keys
    static constexpr int VEC = KW < 4 ? KW : 4;  // words per load
    static constexpr int NV = KW / VEC;
    static constexpr int CPV = VEC * 32 / BITS;  // codes per load
    static constexpr int STEPS = D / 32;         // MFMAs per 16 keys
    static constexpr float kMid = (float)(1 << (BITS - 1));
    struct Tile {
        uint32_t k[2][KW];
        float sk[2], zk[2], w;
    };
};
constexpr int kFewStep = 32 * kWaves;

template <int D, int BITS, bool SYM>
__global__ __launch_bounds__(64 * kWaves, 3) void weigh_few_kernel(WeighArgs a, int cap) {
    using C = Few<D, BITS>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % a.c.heads;
    const int block = blockIdx.x / a.c.heads;
    const int group = a.q_heads / a.c.heads;
    const int shift = a.c.page_shift, ps_mask = (1 << shift) - 1;
    const int pages = (int)a.c.pages;
    const uint32_t k_off = n * C::kRow + g * (C::VEC * 4);
    const uint32_t magic = fp16_magic();

    const Steps<kFewStep> sched(a.batch, shift, lane);
    const int64_t all = sched.total(), share = uniform_div(all + cap - 1, cap);
    const int64_t begin = block * share, end = begin + share < all ? begin + share : all;
    for (int64_t pos = begin; pos < end;) {
        const Place place = sched.at(pos);
        const KvRows &rows = place.rows;
        const int step0 = (int)(pos - place.start);
        const int step1 = end - place.start < place.steps ? (int)(end - place.start) : place.steps;
        pos = place.start + step1;
        const int32_t *const table = a.batch.table + place.seq * a.batch.max_pages;
        const uint32_t total = (uint32_t)rows.n * (uint32_t)group;
        const int kbeg = step0 * kFewStep;
        const int kstop = (int64_t)step1 * kFewStep < rows.len ? step1 * kFewStep : (int)rows.len;
        const int top = (kstop - 1) & ~15;
        const int first_key = kbeg + 32 * wave;
        const int its = kstop > first_key ? (kstop - first_key + kFewStep - 1) / kFewStep : 0;

        // pages of this lane's iteration of the wave, 64 iterations at a time
        int pid0 = 0, pid1 = 0;
        auto load_pages = [&](int it) {
            int k0 = first_key + kFewStep * (it + lane), k1 = k0 + 16;
            k0 = k0 < top ? k0 : top;
            k1 = k1 < top ? k1 : top;
            pid0 = table[k0 >> shift];
            pid1 = table[k1 >> shift];
            asm volatile("" : "+v"(pid0), "+v"(pid1));  // waited for here, not behind later loads
        };
        // One tile of 16 rows, as the launch's rule expects; more of them go
        // over the keys again and add to what the one before has written.
        for (uint32_t tile = 0; tile * 16 < total; ++tile) {
            const float *const before = tile ? a.out : a.weights;
            struct At {
                int64_t slot0, slot1;  // of the tile's two groups of 16 keys
                int key0, key1;        // their first keys; past any key for a page outside the pool
            };
            auto load = [&](typename C::Tile &x, int it) {
                At at;
                if (it > 0 && (it & 63) == 0) load_pages(it);
                const int key0 = first_key + kFewStep * it;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    int page = __builtin_amdgcn_readlane(u ? pid1 : pid0, it & 63);
                    const int key = key0 + 16 * u;
                    const bool in = (uint32_t)page < (uint32_t)pages;
                    (u ? at.key1 : at.key0) = in ? key : 0x7FFFFF00;
                    page = in ? page : 0;
                    const int kc = key < top ? key : top;
                    const int64_t slot = (((int64_t)page * a.c.heads + h) << shift) + (kc & ps_mask);
                    (u ? at.slot1 : at.slot0) = slot;
                    const uint8_t *kp = a.c.k_codes + slot * C::kRow;
#pragma unroll
                    for (int j = 0; j < C::NV; ++j) load_words<C::VEC, true>(x.k[u] + j * C::VEC, kp + j * 64 + k_off);
                    x.sk[u] = a.c.k_scales[slot + n];
                    if (!SYM) x.zk[u] = a.c.k_zeros[slot + n];
                }
                x.w = before ? before[(g & 1 ? at.slot1 : at.slot0) + n] : 0.0f;
                return at;
            };
            typename C::Tile x;
            At at{0, 0, 0, 0};
            if (its > 0) {
                load_pages(0);
                at = load(x, 0);
            }
            // this lane's row as an operand; a row that has seen no key, or a NaN,
            // counts as zeros with a weight of nothing
            const uint32_t rr = tile * 16 + n;
            const bool live = rr < total;
            const uint32_t tok = live ? rr / (uint32_t)group : 0;
            const int qh = h * group + (int)(live ? rr - tok * (uint32_t)group : 0);
            const float lse = live ? a.lse[(rows.begin + tok) * a.q_heads + qh] : __builtin_inff();
            const bool ok = fabsf(lse) < __builtin_inff();
            f16x8 qf[C::STEPS];
            float c1, qsum = 0.0f;
            {
                u32x4 raw[C::STEPS];
                const uint16_t *qp = a.q + (rows.begin + tok) * a.q_stride + (int64_t)qh * D;
#pragma unroll
                for (int s = 0; s < C::STEPS; ++s) {
                    constexpr int SPV = C::CPV / 8;
                    const int d0 = C::CPV * (4 * (s / SPV) + g) + 8 * (s % SPV);
                    raw[s] = ok ? *reinterpret_cast<const u32x4 *>(qp + d0) : u32x4{0u, 0u, 0u, 0u};
                }
                c1 = q_to_fp16<C::STEPS, BITS, SYM, false>(raw, a.scale, qf, qsum);
                if (!SYM) qsum = add_halves16(add_halves32(qsum));
            }
            // rows 4 g + i of the products
            const float minus = ok ? -lse * kLog2e : -__builtin_inff();
            const int mine = live ? (int)(rows.first + tok) : -1;  // last position the row sees
            float c1r[4], nl[4], qs[4];
            int last[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c1r[i] = __shfl(c1, 4 * g + i);
                nl[i] = __shfl(minus, 4 * g + i);
                last[i] = __shfl(mine, 4 * g + i);
                if (!SYM) qs[i] = __shfl(qsum, 4 * g + i);
            }
            const int safe = (int)(rows.first + tile * 16 / (uint32_t)group);  // every row sees up to here

            for (int it = 0; it < its; ++it) {
                f32x4 t[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    t[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < C::STEPS; ++s) {
                        f16x2 kf[4];
                        if constexpr (BITS == 8) {
                            int8_row(x.k[u][2 * s], kf);
                            int8_row(x.k[u][2 * s + 1], kf + 2);
                        } else {
                            const uint32_t w = x.k[u][s], w8 = w >> 8;
                            kf[0] = int4_low(w, magic); kf[1] = int4_high(w, magic);
                            kf[2] = int4_low(w8, magic); kf[3] = int4_high(w8, magic);
                        }
                        t[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(qf[s], join(kf), t[u], 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (!SYM) t[u][i] = __builtin_fmaf(C::kMid - x.zk[u], qs[i], t[u][i]);
                        t[u][i] *= x.sk[u];
                    }
                }
                const int k0 = at.key0 + n, k1 = at.key1 + n, key = g & 1 ? k1 : k0;
                const int64_t slot = (g & 1 ? at.slot1 : at.slot0) + n;
                const bool masked = at.key0 + 15 > safe || at.key1 + 15 > safe;
                const float was = key < rows.first || tile ? x.w : 0.0f;  // the call's own tokens start from nothing
                if (it + 1 < its) at = load(x, it + 1);
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t[u][i], c1r[i], nl[i]));
                        if (masked) p = (u ? k1 : k0) > last[i] ? 0.0f : p;
                        sum[u] += p;
                    }
                sum[0] = add_halves32(add_halves16(sum[0]));
                sum[1] = add_halves32(add_halves16(sum[1]));
                if (g < 2 && key < kstop) a.out[slot] = was + (g ? sum[1] : sum[0]);
            }
        }
    }
}

// ---- many rows: KT keys in a block's registers, rows streamed past them ----
//
// The codes less their zeros are integers of up to 9 bits, which bf16 holds
// exactly, so the rows are multiplied as they lie. The block turns the codes
// into operands once, through LDS, and all four waves keep all of them; wave w
// takes the row tiles w, w + 4, ..., the next one's loads in flight.
template <int D, int BITS, int KT>
struct Many {
    static constexpr int kRow = D * BITS / 8;
    static constexpr int TPK = 64 * kWaves / KT;     // threads a key
    static constexpr int PIECES = D / TPK / 8;       // operands of 8 codes a thread
    static constexpr int WORDS = kRow / TPK / 4;     // code words a thread
    static constexpr int S = D / 32;                 // MFMAs per 16 keys
    static constexpr int TILES = KT / 16;
    static constexpr float kMid = (float)(1 << (BITS - 1));
    struct Rows {
        u32x4 raw[S];
        float lse;
    };
};

template <int D, int BITS, bool SYM, int KT>
__global__ __launch_bounds__(64 * kWaves, 2) void weigh_many_kernel(WeighArgs a, int cap) {
    using C = Many<D, BITS, KT>;
    __shared__ bf16x8 ops[C::TILES][C::S][64];
    __shared__ float key_scale[KT], rest[KT], part[kWaves][KT];
    __shared__ int64_t slots[KT];  // -1: not a key
    __shared__ int wide;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % a.c.heads;
    const int group = a.q_heads / a.c.heads;
    const int shift = a.c.page_shift, ps_mask = (1 << shift) - 1;
    const int my_key = threadIdx.x / C::TPK, my_part = threadIdx.x % C::TPK;
    const uint32_t dtok = 16 * kWaves / (uint32_t)group, drem = 16 * kWaves % (uint32_t)group;

    const Steps<KT> sched(a.batch, shift, lane);
    const int64_t all = sched.total();
    for (int64_t pos = blockIdx.x / a.c.heads; pos < all; pos += cap) {
        const Place place = sched.at(pos);
        const KvRows &rows = place.rows;
        const int32_t *const table = a.batch.table + place.seq * a.batch.max_pages;
        const int k0 = (int)(pos - place.start) * KT;
        const uint32_t total = (uint32_t)rows.n * (uint32_t)group;
        // rows before the first key see none of them
        const int64_t late = k0 - rows.first;
        const uint32_t row0 = late <= 0 ? 0 : late < rows.n ? (uint32_t)late * (uint32_t)group : total;
        const uint32_t tile0 = row0 / 16, tiles = (total + 15) / 16;

        if (threadIdx.x == 0) wide = 0;
        __syncthreads();  // nobody reads the last step's keys any more
        {
            const int key = k0 + my_key, kc = key < rows.len ? key : (int)rows.len - 1;
            int64_t page = table[kc >> shift];
            const bool in = key < rows.len && page >= 0 && page < a.c.pages;
            page = in ? page : 0;
            const int64_t slot = ((page * a.c.heads + h) << shift) + (kc & ps_mask);
            const uint32_t *src = reinterpret_cast<const uint32_t *>(a.c.k_codes + slot * C::kRow) + my_part * C::WORDS;
            uint32_t w[C::WORDS];
#pragma unroll
            for (int i = 0; i < C::WORDS; i += 4) {
                if constexpr (C::WORDS >= 4) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(src + i);
                    w[i] = v[0]; w[i + 1] = v[1]; w[i + 2] = v[2]; w[i + 3] = v[3];
                } else if constexpr (C::WORDS == 2) {
                    const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
                    w[0] = v[0]; w[1] = v[1];
                } else {
                    w[0] = src[0];
                }
            }
            float near = C::kMid, left = 0.0f;
            if (!SYM) {
                const float z = in ? a.c.k_zeros[slot] : 0.0f;
                near = fminf(fmaxf(rintf(z), 0.0f), 2.0f * C::kMid - 1.0f);
                left = z - near;
                if (left != 0.0f) wide = 1;
            }
            if (my_part == 0) {
                slots[my_key] = in ? slot : -1;
                key_scale[my_key] = in ? a.c.k_scales[slot] * (a.scale * kLog2e) : 0.0f;
                rest[my_key] = left;
            }
#pragma unroll
            for (int i = 0; i < C::PIECES; ++i) {
                bf16x8 f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t c = BITS == 8 ? (w[(2 * i + e / 4) % C::WORDS] >> (8 * (e % 4))) & 255u
                                                 : (w[i % C::WORDS] >> (4 * e)) & 15u;
                    f[e] = (__bf16)((float)c - near);
                }
                const int e0 = my_part * (D / C::TPK) + 8 * i;
                ops[my_key / 16][e0 / 32][(e0 % 32) / 8 * 16 + my_key % 16] = f;
            }
        }
        __syncthreads();
        bf16x8 kf[C::TILES][C::S];
        float cs[C::TILES], acc[C::TILES];
#pragma unroll
        for (int k = 0; k < C::TILES; ++k) {
            cs[k] = key_scale[16 * k + n];
            acc[k] = 0.0f;
#pragma unroll
            for (int s = 0; s < C::S; ++s) kf[k][s] = ops[k][s][lane];
        }
        const bool any_wide = !SYM && wide;

        // the lane's row as an operand, and its way to the wave's next tile
        uint32_t rr = (tile0 + wave) * 16 + n;
        uint32_t tok = rr / (uint32_t)group, rem = rr - tok * (uint32_t)group;
        auto load = [&](typename C::Rows &x) {
            const bool live = rr < total;
            const int64_t row = rows.begin + (live ? tok : 0);
            const int qh = h * group + (live ? (int)rem : 0);
            x.lse = live ? a.lse[row * a.q_heads + qh] : __builtin_inff();
            const uint16_t *qp = a.q + row * a.q_stride + (int64_t)qh * D + 8 * g;
#pragma unroll
            for (int s = 0; s < C::S; ++s)
                x.raw[s] = live ? *reinterpret_cast<const u32x4 *>(qp + 32 * s) : u32x4{0u, 0u, 0u, 0u};
        };
        typename C::Rows x;
        if (tile0 + wave < tiles) load(x);
        for (uint32_t tile = tile0 + wave; tile < tiles; tile += kWaves) {
            bf16x8 qf[C::S];
            // a row that has seen no key, or a NaN, counts as zeros with a weight of nothing
            const bool ok = fabsf(x.lse) < __builtin_inff();
            const float minus = ok ? -x.lse * kLog2e : -__builtin_inff();
            if (__any(!ok)) {
#pragma unroll
                for (int s = 0; s < C::S; ++s) x.raw[s] = ok ? x.raw[s] : u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int s = 0; s < C::S; ++s) qf[s] = __builtin_bit_cast(bf16x8, x.raw[s]);
            float nl[4], qs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) nl[i] = __shfl(minus, 4 * g + i);
            if (any_wide) {
                f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
                bf16x8 ones;
#pragma unroll
                for (int e = 0; e < 8; ++e) ones[e] = (__bf16)1.0f;
#pragma unroll
                for (int s = 0; s < C::S; ++s) v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[s], ones, v, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) qs[i] = v[i];
            }
            const int64_t sees = rows.first + tok;
            // keys that some row of the tile does not see
            const bool masked = k0 + KT - 1 > __builtin_amdgcn_readfirstlane((int)sees);
            int last[4] = {0, 0, 0, 0};
            if (masked) {
#pragma unroll
                for (int i = 0; i < 4; ++i) last[i] = __shfl((int)sees, 4 * g + i);
            }
            rr += 16 * kWaves;
            tok += dtok;
            rem += drem;
            if (rem >= (uint32_t)group) {
                rem -= group;
                ++tok;
            }
            if (tile + kWaves < tiles) load(x);
#pragma unroll
            for (int k = 0; k < C::TILES; ++k) {
                f32x4 t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < C::S; ++s) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[s], kf[k][s], t, 0, 0, 0);
                if (any_wide) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i] = __builtin_fmaf(-rest[16 * k + n], qs[i], t[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t[i], cs[k], nl[i]));
                    if (masked) p = k0 + 16 * k + n > last[i] ? 0.0f : p;
                    acc[k] += p;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < C::TILES; ++k) {
            acc[k] = add_halves32(add_halves16(acc[k]));
            if (g == 0) part[wave][16 * k + n] = acc[k];
        }
        __syncthreads();
        if (threadIdx.x < KT && slots[threadIdx.x] >= 0) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) sum += part[w][threadIdx.x];
            // the call's own tokens start from nothing
            const int64_t slot = slots[threadIdx.x];
            const bool old = a.weights && k0 + (int)threadIdx.x < rows.first;
            a.out[slot] = (old ? a.weights[slot] : 0.0f) + sum;
        }
    }
}

}  // namespace

template <int D, int BITS, bool SYM>
static hipError_t launch(const WeighArgs &a, hipStream_t st) {
    const int64_t group = a.q_heads / a.c.heads, heads = a.c.heads, b = a.batch.b;
    const int64_t room = a.batch.max_pages << a.c.page_shift;
    const int64_t n = a.max_rows <= 0 || a.max_rows > a.batch.rows ? a.batch.rows : a.max_rows;
    const int64_t kv = a.max_kv <= 0 || a.max_kv > room ? room : a.max_kv;
    // blocks a key head: no more than steps of work, nor than `most` in all
    auto blocks = [&](int64_t step, int64_t most) {
        const int64_t steps = b * ((kv + step - 1) / step < 1 ? 1 : (kv + step - 1) / step);
        const int64_t cap = (most + heads - 1) / heads;
        return (int)(cap < steps ? cap : steps);
    };
    if (n * group <= 16) {
        const int cap = blocks(kFewStep, 768);
        hipLaunchKernelGGL((weigh_few_kernel<D, BITS, SYM>), dim3((uint32_t)(cap * heads)), dim3(64 * kWaves), 0, st, a, cap);
        return hipGetLastError();
    }
    constexpr int KT = D == 256 ? 64 : 128;
    if (blocks(KT, 1 << 20) * heads >= 512) {
        const int cap = blocks(KT, 1 << 16);
        hipLaunchKernelGGL((weigh_many_kernel<D, BITS, SYM, KT>), dim3((uint32_t)(cap * heads)), dim3(64 * kWaves), 0, st, a, cap);
    } else {
        const int cap = blocks(32, 1 << 16);
        hipLaunchKernelGGL((weigh_many_kernel<D, BITS, SYM, 32>), dim3((uint32_t)(cap * heads)), dim3(64 * kWaves), 0, st, a, cap);
    }
    return hipGetLastError();
}

hipError_t launch_kv_weigh(const WeighArgs &a, hipStream_t st) {
#define LQ_WEIGH(D, BITS, SYM) \
    if (a.c.head_dim == D && a.c.bits == BITS && (a.c.symmetric != 0) == SYM) return launch<D, BITS, SYM>(a, st);
#define LQ_WEIGH_D(D) LQ_WEIGH(D, 4, false) LQ_WEIGH(D, 4, true) LQ_WEIGH(D, 8, false) LQ_WEIGH(D, 8, true)
    LQ_WEIGH_D(64) LQ_WEIGH_D(128) LQ_WEIGH_D(256)
#undef LQ_WEIGH_D
#undef LQ_WEIGH
    return hipErrorInvalidValue;
}

}  // namespace lq
