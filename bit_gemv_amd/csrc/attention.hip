// attention.hip -- causal attention of new tokens over the quantized paged
// cache (paged_attention).
//
// With codes c, scale s and zero z of a key or value, x_hat = s (c - z):
//   score_ij = s_j (q_i . c_j - z_j sum(q_i))
//   o_i      = sum_j p_ij s_j (c_j - z_j) / sum_j p_ij,  p = exp(score - max)
// so both products take the codes as they are. Codes become exact fp16
// integers (c - 2^(bits-1)) by placing their bits in the mantissa of 1024 and
// subtracting; q becomes fp16 exactly after a power-of-two scaling; the key
// scale is applied to the fp32 score and the value scale to p before it is
// rounded to fp16 (2^-11), normalized by a running bound of the value scales
// so that it stays in fp16's range.
//
// The first product is formed transposed, keys x rows: a lane then holds four
// neighbouring keys of one row, which is the operand layout that the second
// product (again transposed, elements x rows) wants of p, with no exchange
// between lanes; maximum, sum and rescaling are per lane.
#include "common.hpp"
#include "kv.hpp"

namespace lq {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
// p is taken relative to a running reference of the row's maximum that is
// raised only when a score passes it by kSlack (in log2), and the value
// scale relative to a reference raised when one passes it 2^6-fold: fp16
// weights stay at most 2^3 2^6 2^6 = 2^15, and everything down to 2^-28 of
// the largest keeps a nonzero weight.
constexpr float kSlack = 6.0f;
constexpr float kScaleSlack = 64.0f;
constexpr float kHead = 8.0f;

// fp16 pairs of a code word, minus the middle code: INT8 bytes (0, 1), (2, 3)
// or (0, 2), (1, 3); INT4 nibbles (0, 4), (1, 5), (2, 6), (3, 7). A code in
// the low mantissa bits of fp16 1024 is 1024 + c, one four bits higher
// 1024 + 16 c; both differences are exact.
LQ_DEVICE f16x2 as_f16x2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }

LQ_DEVICE void int8_pairs(uint32_t w, uint32_t sel0, uint32_t sel1, f16x2 *out) {
    const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
    out[0] = as_f16x2(__builtin_amdgcn_perm(0x64646464u, w, sel0)) - off;
    out[1] = as_f16x2(__builtin_amdgcn_perm(0x64646464u, w, sel1)) - off;
}
LQ_DEVICE f16x2 int4_low(uint32_t w) {
    const f16x2 off = {(_Float16)1032.0f, (_Float16)1032.0f};
    return as_f16x2((w & 0x000F000Fu) | 0x64006400u) - off;
}
LQ_DEVICE f16x2 int4_high(uint32_t w) {
    const f16x2 sc = {(_Float16)0.0625f, (_Float16)0.0625f}, off = {(_Float16)-72.0f, (_Float16)-72.0f};
    return __builtin_elementwise_fma(as_f16x2((w & 0x00F000F0u) | 0x64006400u), sc, off);
}

LQ_DEVICE f16x8 join(const f16x2 *p) {
    return f16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

LQ_DEVICE float max_halves32(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
LQ_DEVICE float max_halves16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Where a block writes: the output itself, or one split's partial result
// (o unnormalized relative to the split's maximum, log2 units).
struct Partials {
    float *o;   // [splits][rows][q_heads][D]
    float *ml;  // [splits][rows][q_heads][2]
    int splits;
};

// ---- few rows: one wave per run of 32 keys, no sharing between waves ----
//
// A block of four waves takes one (sequence, key head, 16 query rows, split);
// its rows are the heads of the group, token by token. Wave w walks the
// split's 32-key tiles w, w + 4, ... with the next tile's codes and scales in
// flight; the waves' results are joined in LDS.
template <int D, int BITS, bool SYM>
struct Few {
    static constexpr int kRow = D * BITS / 8;        // code bytes of a token
    static constexpr int KW = D * BITS / 128;        // code words per lane of 16 keys
    static constexpr int VEC = KW < 4 ? KW : 4;      // words per load
    static constexpr int NV = KW / VEC;              // loads
    static constexpr int CPV = VEC * 32 / BITS;      // codes per load
    static constexpr int STEPS = D / 32;             // score MFMAs per 16 keys
    static constexpr int TILES = D / 16;             // output MFMA tiles
    static constexpr float kMid = (float)(1 << (BITS - 1));

    struct Tile {
        uint32_t k[2][KW], v[2][KW];
        f32x4 sk[2], sv[2], zk[2], zv[2];
        int64_t key[2];  // first key of the 16, or past everything for a page outside the pool
    };
};

template <int N>
LQ_DEVICE void load_words(uint32_t *dst, const uint8_t *p) {
    if constexpr (N == 4) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
        dst[0] = v[0]; dst[1] = v[1]; dst[2] = v[2]; dst[3] = v[3];
    } else {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
        dst[0] = v[0]; dst[1] = v[1];
    }
}

template <int D, int BITS, bool SYM>
__global__ __launch_bounds__(256, 2) void attn_few_kernel(AttnArgs a, Partials part, int grid_tiles) {
    using C = Few<D, BITS, SYM>;
    constexpr int LDO = D + 4;
    __shared__ float lds_o[4][16][LDO];
    __shared__ float lds_m[4][16], lds_l[4][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % a.c.heads;
    const int split = (blockIdx.x / a.c.heads) % part.splits;
    const int tile0 = blockIdx.x / a.c.heads / part.splits;
    const int group = a.q_heads / a.c.heads;
    const int ps_mask = (1 << a.c.page_shift) - 1;
    const int64_t seq = blockIdx.y;
    {
        const KvRows rows = kv_rows(a.batch, seq, a.c.page_shift);
        const int64_t total = rows.n * group;
        for (int64_t tile = tile0; tile * 16 < total; tile += grid_tiles) {
            // this lane's query row
            const int64_t rr = tile * 16 + n;
            const bool live = rr < total;
            const int64_t tok = live ? rr / group : 0;
            const int qh = h * group + (int)(live ? rr % group : 0);
            const int64_t last_row = (tile * 16 + 15 < total ? tile * 16 + 15 : total - 1) / group;
            const int64_t row_pos = live ? rows.first + tok : -1;   // last position the row sees
            const int64_t safe = rows.first + tile * 16 / group;    // every row sees up to here
            int64_t kend = rows.first + last_row + 1;
            if (kend > rows.len) kend = rows.len;
            if (kend < 0) kend = 0;
            const int64_t per = ((kend + part.splits - 1) / part.splits + 127) / 128 * 128;
            const int64_t kbeg = split * per;
            const int64_t kstop = kbeg + per < kend ? kbeg + per : kend;

            // q, its scaling to fp16 and the sum of its elements
            f16x8 qf[C::STEPS];
            float unscale, qsum = 0.0f;
            {
                u32x4 raw[C::STEPS];
                const uint16_t *qp = a.q + (rows.begin + tok) * a.q_stride + (int64_t)qh * D;
                float amax = 0.0f;
#pragma unroll
                for (int s = 0; s < C::STEPS; ++s) {
                    constexpr int SPV = C::CPV / 8;
                    const int d0 = C::CPV * (4 * (s / SPV) + g) + 8 * (s % SPV);
                    raw[s] = live ? *reinterpret_cast<const u32x4 *>(qp + d0) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[s][j])), fabsf(bf16_hi(raw[s][j]))));
                }
                amax = team_max<64>(amax);
                int sh = 137 - (int)(__float_as_uint(amax) >> 23);  // the largest into [2^10, 2^11)
                sh = sh < -117 ? -117 : sh > 100 ? 100 : sh;
                const float up = __uint_as_float((uint32_t)(sh + 127) << 23);
                unscale = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
                for (int s = 0; s < C::STEPS; ++s) {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f[2 * j] = bf16_lo(raw[s][j]) * up;
                        f[2 * j + 1] = bf16_hi(raw[s][j]) * up;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // INT4 words come out as nibbles 0 4 1 5 2 6 3 7
                        const int src = BITS == 8 ? e : (e >> 1) + 4 * (e & 1);
                        qf[s][e] = (_Float16)f[src];
                        if (!SYM) qsum += (float)qf[s][e];
                    }
                }
                if (!SYM) {
                    qsum += __shfl_xor(qsum, 16, 64);
                    qsum += __shfl_xor(qsum, 32, 64);
                }
            }
            const float c1 = a.scale * kLog2e * unscale;

            f32x4 o[C::TILES];
#pragma unroll
            for (int t = 0; t < C::TILES; ++t) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            float m = -1e30f, l = 0.0f, vz = 0.0f, sref = 0.0f, inv_sref = 0.0f;

            int pid0 = 0, pid1 = 0;  // pages of this lane's iteration of the wave, 64 at a time
            auto load_tile = [&](typename C::Tile &x, int it) {
                const int64_t key0 = kbeg + 32 * (int64_t)(wave + 4 * it);
                if ((it & 63) == 0) {
                    const int64_t top = (kstop - 1) & ~(int64_t)15;
                    int64_t k0 = key0 + 128 * (int64_t)lane, k1 = k0 + 16;
                    k0 = k0 < top ? k0 : top;
                    k1 = k1 < top ? k1 : top;
                    pid0 = a.batch.table[seq * a.batch.max_pages + (k0 >> a.c.page_shift)];
                    pid1 = a.batch.table[seq * a.batch.max_pages + (k1 >> a.c.page_shift)];
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    int page = __builtin_amdgcn_readlane(u ? pid1 : pid0, it & 63);
                    const int64_t key = key0 + 16 * u;
                    const bool in = page >= 0 && page < a.c.pages;
                    x.key[u] = in ? key : (int64_t)1 << 60;
                    page = in ? page : 0;
                    const int64_t top = (kstop - 1) & ~(int64_t)15;
                    const int64_t kc = key < top ? key : top;
                    const int64_t slot = (((int64_t)page * a.c.heads + h) << a.c.page_shift) + (kc & ps_mask);
                    const uint8_t *kp = a.c.k_codes + (slot + n) * C::kRow + g * (C::VEC * 4);
                    const uint8_t *vp = a.c.v_codes + (slot + 4 * g) * C::kRow + n * (C::VEC * 4);
#pragma unroll
                    for (int j = 0; j < C::NV; ++j) load_words<C::VEC>(x.k[u] + j * C::VEC, kp + j * 64);
#pragma unroll
                    for (int j = 0; j < C::NV; ++j) load_words<C::VEC>(x.v[u] + j * C::VEC, vp + j * 256);
                    x.sk[u] = *reinterpret_cast<const f32x4 *>(a.c.k_scales + slot + 4 * g);
                    x.sv[u] = *reinterpret_cast<const f32x4 *>(a.c.v_scales + slot + 4 * g);
                    if (!SYM) {
                        x.zk[u] = *reinterpret_cast<const f32x4 *>(a.c.k_zeros + slot + 4 * g);
                        x.zv[u] = *reinterpret_cast<const f32x4 *>(a.c.v_zeros + slot + 4 * g);
                    }
                }
            };
            auto use_tile = [&](typename C::Tile &x) {
                f32x4 acc[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    acc[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < C::STEPS; ++s) {
                        f16x2 kf[4];
                        if constexpr (BITS == 8) {
                            int8_pairs(x.k[u][2 * s], 0x04010400u, 0x04030402u, kf);
                            int8_pairs(x.k[u][2 * s + 1], 0x04010400u, 0x04030402u, kf + 2);
                        } else {
                            const uint32_t w = x.k[u][s], w8 = w >> 8;
                            kf[0] = int4_low(w); kf[1] = int4_high(w);
                            kf[2] = int4_low(w8); kf[3] = int4_high(w8);
                        }
                        acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(kf), qf[s], acc[u], 0, 0, 0);
                    }
                }
                float t[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float ak = x.sk[u][i] * c1;
                        t[u][i] = SYM ? acc[u][i] * ak : (acc[u][i] - (x.zk[u][i] - C::kMid) * qsum) * ak;
                    }
                if (x.key[0] + 15 > safe || x.key[1] + 15 > safe || x.key[1] + 15 >= kstop) {
                    // keys some row does not see, or nobody: they may hold anything
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int64_t key = x.key[u] + 4 * g + i;
                            if (key > row_pos || key >= kstop) t[u][i] = -__builtin_inff();
                            if (key >= kstop) {
                                x.sv[u][i] = 0.0f;
                                if (!SYM) x.zv[u][i] = 0.0f;
                            }
                        }
                }
                float tm = fmaxf(fmaxf(fmaxf(t[0][0], t[0][1]), fmaxf(t[0][2], t[0][3])),
                                 fmaxf(fmaxf(t[1][0], t[1][1]), fmaxf(t[1][2], t[1][3])));
                float sm = fmaxf(fmaxf(fmaxf(x.sv[0][0], x.sv[0][1]), fmaxf(x.sv[0][2], x.sv[0][3])),
                                 fmaxf(fmaxf(x.sv[1][0], x.sv[1][1]), fmaxf(x.sv[1][2], x.sv[1][3])));
                if (__any(tm > m + kSlack || sm > sref * kScaleSlack)) {
                    tm = max_halves16(max_halves32(tm));
                    sm = max_halves16(max_halves32(sm));
                    const float mn = fmaxf(m, tm), sn = fmaxf(sref, sm);
                    const float down = __builtin_amdgcn_exp2f(m - mn);
                    const float both = sn > 0.0f ? down * (sref / sn) : 1.0f;
                    l *= down;
                    vz *= both;
#pragma unroll
                    for (int q = 0; q < C::TILES; ++q) o[q] *= both;
                    m = mn;
                    sref = sn;
                    inv_sref = kHead / fmaxf(sn, 1e-30f);
                }
                f16x2 pb[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float pv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = __builtin_amdgcn_exp2f(t[u][i] - m);
                        l += p;
                        pv[i] = p * (x.sv[u][i] * inv_sref);
                    }
                    pb[2 * u] = f16x2{(_Float16)pv[0], (_Float16)pv[2]};
                    pb[2 * u + 1] = f16x2{(_Float16)pv[1], (_Float16)pv[3]};
                    if (!SYM) {
                        // the zero's share, from the same rounded weights
                        vz += (float)pb[2 * u][0] * (x.zv[u][0] - C::kMid);
                        vz += (float)pb[2 * u][1] * (x.zv[u][2] - C::kMid);
                        vz += (float)pb[2 * u + 1][0] * (x.zv[u][1] - C::kMid);
                        vz += (float)pb[2 * u + 1][1] * (x.zv[u][3] - C::kMid);
                    }
                }
                const f16x8 pf = join(pb);
#pragma unroll
                for (int w = 0; w < C::KW; ++w) {
                    f16x2 vf[4];
                    if constexpr (BITS == 8) {
                        int8_pairs(x.v[0][w], 0x04020400u, 0x04030401u, vf);
                        int8_pairs(x.v[1][w], 0x04020400u, 0x04030401u, vf + 2);
                        o[w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(vf), pf, o[w], 0, 0, 0);
                    } else {
                        const uint32_t v0 = x.v[0][w], v1 = x.v[1][w];
                        vf[0] = int4_low(v0); vf[1] = int4_low(v0 >> 8);
                        vf[2] = int4_low(v1); vf[3] = int4_low(v1 >> 8);
                        o[2 * w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(vf), pf, o[2 * w], 0, 0, 0);
                        vf[0] = int4_high(v0); vf[1] = int4_high(v0 >> 8);
                        vf[2] = int4_high(v1); vf[3] = int4_high(v1 >> 8);
                        o[2 * w + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(vf), pf, o[2 * w + 1], 0, 0, 0);
                    }
                }
            };

            const int its = kstop > kbeg + 32 * wave ? (int)((kstop - kbeg - 32 * wave + 127) / 128) : 0;
            if (its > 0) {
                typename C::Tile x, y;
                load_tile(x, 0);
                for (int it = 0; it < its; it += 2) {
                    if (it + 1 < its) load_tile(y, it + 1);
                    use_tile(x);
                    if (it + 1 < its) {
                        if (it + 2 < its) load_tile(x, it + 2);
                        use_tile(y);
                    }
                }
            }
            l += __shfl_xor(l, 16, 64);
            l += __shfl_xor(l, 32, 64);
            if (!SYM) {
                vz += __shfl_xor(vz, 16, 64);
                vz += __shfl_xor(vz, 32, 64);
            }

            // join the four waves
            if (g == 0) {
                lds_m[wave][n] = m;
                lds_l[wave][n] = l;
            }
            __syncthreads();
            const float mall = fmaxf(fmaxf(lds_m[0][n], lds_m[1][n]), fmaxf(lds_m[2][n], lds_m[3][n]));
            const float f = __builtin_amdgcn_exp2f(m - mall) * (sref * (1.0f / kHead));
#pragma unroll
            for (int j = 0; j < C::NV; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // elements of word t of load j in matrix row 4 g + i
                    constexpr int EPW = 8 / BITS;
                    float *dst = &lds_o[wave][n][((j * 16 + 4 * g + i) * C::VEC) * EPW];
#pragma unroll
                    for (int t = 0; t < C::VEC * EPW; ++t) dst[t] = (o[j * C::VEC * EPW + t][i] - vz) * f;
                }
            __syncthreads();
            {
                const int r = threadIdx.x >> 4, c = threadIdx.x & 15;
                const int64_t wr = tile * 16 + r;
                if (wr < total) {
                    const float mr = fmaxf(fmaxf(lds_m[0][r], lds_m[1][r]), fmaxf(lds_m[2][r], lds_m[3][r]));
                    float lr = 0.0f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) lr += lds_l[w][r] * __builtin_amdgcn_exp2f(lds_m[w][r] - mr);
                    const int64_t at = (rows.begin + wr / group) * a.q_heads + h * group + wr % group;
                    const float norm = part.splits > 1 ? 1.0f : lr > 0.0f ? 1.0f / lr : 0.0f;
#pragma unroll
                    for (int d = 4 * c; d < D; d += 64) {
                        f32x4 v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int w = 0; w < 4; ++w) v += *reinterpret_cast<const f32x4 *>(&lds_o[w][r][d]);
                        v *= norm;
                        if (part.splits > 1) {
                            if (lr > 0.0f)
                                *reinterpret_cast<f32x4 *>(
                                    part.o + ((int64_t)split * a.batch.rows * a.q_heads + at) * D + d) = v;
                        } else {
                            const bf16x2_t b0{(__bf16)v[0], (__bf16)v[1]}, b1{(__bf16)v[2], (__bf16)v[3]};
                            *reinterpret_cast<u32x2 *>(a.out + at * D + d) =
                                u32x2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
                        }
                    }
                    if (c == 0) {
                        if (part.splits > 1) {
                            float *ml = part.ml + ((int64_t)split * a.batch.rows * a.q_heads + at) * 2;
                            ml[0] = lr > 0.0f ? mr : -__builtin_inff();
                            ml[1] = lr;
                        } else if (a.lse) {
                            a.lse[at] = lr > 0.0f ? mr * kLn2 + logf(lr) : -__builtin_inff();
                        }
                    }
                }
            }
            __syncthreads();  // the next row tile reuses the buffers
        }
    }
}

// Joins the splits of each (row, head): D / 4 lanes each.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Partials part) {
    constexpr int W = D / 4;
    const int64_t at = (int64_t)blockIdx.x * (256 / W) + threadIdx.x / W;
    const int c = threadIdx.x % W;
    const int64_t all = a.batch.rows * a.q_heads;
    int64_t lo = a.batch.starts[0], hi = a.batch.starts[a.batch.b];
    const int64_t row = at / a.q_heads;
    if (at >= all || row < lo || row >= hi) return;
    float m = -1e30f;
    for (int s = 0; s < part.splits; ++s) m = fmaxf(m, part.ml[(s * all + at) * 2]);
    float l = 0.0f;
    f32x4 v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < part.splits; ++s) {
        const float ms = part.ml[(s * all + at) * 2];
        if (ms == -__builtin_inff()) continue;  // nothing seen there: no partial was written
        const float f = __builtin_amdgcn_exp2f(ms - m);
        l += f * part.ml[(s * all + at) * 2 + 1];
        v += *reinterpret_cast<const f32x4 *>(part.o + (s * all + at) * D + 4 * c) * f;
    }
    const float norm = l > 0.0f ? 1.0f / l : 0.0f;
    v *= norm;
    const bf16x2_t b0{(__bf16)v[0], (__bf16)v[1]}, b1{(__bf16)v[2], (__bf16)v[3]};
    *reinterpret_cast<u32x2 *>(a.out + at * D + 4 * c) =
        u32x2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
    if (c == 0 && a.lse) a.lse[at] = l > 0.0f ? m * kLn2 + logf(l) : -__builtin_inff();
}

struct Plan {
    int splits;
    int64_t tiles;  // row tiles of a sequence
    int64_t bytes;
};

Plan plan_of(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t b, int64_t room, int64_t max_rows,
             int64_t max_kv) {
    Plan p;
    const int64_t n = max_rows <= 0 || max_rows > rows ? rows : max_rows;
    const int64_t kv = max_kv <= 0 || max_kv > room ? room : max_kv;
    p.tiles = (n * (q_heads / heads) + 15) / 16;
    const int64_t blocks = b * heads * p.tiles;
    int64_t s = (1024 + blocks - 1) / blocks;
    const int64_t most = (kv + 127) / 128;
    if (s > most) s = most;
    if (s > 128) s = 128;
    p.splits = s < 1 ? 1 : (int)s;
    p.bytes = p.splits > 1 ? p.splits * rows * q_heads * (head_dim + 2) * 4 : 0;
    return p;
}

}  // namespace

int64_t attention_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t b,
                                  int64_t max_pages, int64_t page_size, int64_t max_rows, int64_t max_kv) {
    return plan_of(rows, q_heads, heads, head_dim, b, max_pages * page_size, max_rows, max_kv).bytes;
}

template <int D, int BITS, bool SYM>
static hipError_t launch_few(const AttnArgs &a, const Plan &p, hipStream_t st) {
    Partials part{static_cast<float *>(a.workspace), nullptr, p.splits};
    part.ml = part.o + (int64_t)p.splits * a.batch.rows * a.q_heads * D;
    int64_t tiles = p.tiles;
    const int64_t per_tile = (int64_t)p.splits * a.c.heads;
    if (tiles * per_tile > 1 << 30) tiles = (1 << 30) / per_tile;
    const dim3 grid((uint32_t)(tiles * per_tile), (uint32_t)a.batch.b);
    hipLaunchKernelGGL((attn_few_kernel<D, BITS, SYM>), grid, dim3(256), 0, st, a, part, (int)tiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t pairs = a.batch.rows * a.q_heads, per = 256 / (D / 4);
    hipLaunchKernelGGL((attn_join_kernel<D>), dim3((uint32_t)((pairs + per - 1) / per)), dim3(256), 0, st, a, part);
    return hipGetLastError();
}

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st) {
    const Plan p = plan_of(a.batch.rows, a.q_heads, a.c.heads, a.c.head_dim, a.batch.b,
                           a.batch.max_pages << a.c.page_shift, a.max_rows, a.max_kv);
#define LQ_ATTN(D, BITS, SYM) \
    if (a.c.head_dim == D && a.c.bits == BITS && (a.c.symmetric != 0) == SYM) return launch_few<D, BITS, SYM>(a, p, st);
#define LQ_ATTN_D(D) LQ_ATTN(D, 4, false) LQ_ATTN(D, 4, true) LQ_ATTN(D, 8, false) LQ_ATTN(D, 8, true)
    LQ_ATTN_D(64) LQ_ATTN_D(128) LQ_ATTN_D(256)
#undef LQ_ATTN_D
#undef LQ_ATTN
    return hipErrorInvalidValue;
}

}  // namespace lq
