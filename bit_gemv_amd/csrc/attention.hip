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
// so that it stays in fp16's range. A value zero outside the codes counts with
// the unrounded p: its weight may vanish in fp16 while scale times zero is large.
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
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
// p is taken relative to a running reference of the row's maximum that is
// raised only when a score passes it by kSlack (in log2), and the value
// scale relative to a reference raised when one passes it 2^6-fold: fp16
// weights stay at most 2^3 2^6 2^6 = 2^15, and everything down to 2^-28 of
// the largest keeps a nonzero weight.
constexpr float kSlack = 6.0f;
constexpr float kScaleSlack = 64.0f;
constexpr float kScaleMin = 9.094947017729282e-13f;  // 2^-40, below every scale kv_cache_write makes
constexpr float kHead = 8.0f, kHeadLog2 = 3.0f;

// Codes as fp16 pairs less the middle code, exactly: a code in the low mantissa
// bits of fp16 1024 is 1024 + c, one four bits higher 1024 + 16 c. INT8 pairs
// are bytes (0, 1), (2, 3) or (0, 2), (1, 3); INT4 pairs nibbles (0, 4), (1, 5)
// of a word and the same of the word shifted by 8. (Raw codes as fp16
// subnormals, which the matrix instructions take exactly, would save the
// subtraction, a quarter of the conversion; but the sums then carry the middle
// code, and the matrix instructions' rounding of them moved scores of 25 by
// 3e-5 where this form stays within 1e-6, and would bias long sums of values.)
LQ_DEVICE f16x2 as_f16x2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }

template <uint32_t SEL0, uint32_t SEL1>
LQ_DEVICE void int8_pairs(uint32_t w, f16x2 *out, f16x2 off0, f16x2 off1) {
    out[0] = as_f16x2(__builtin_amdgcn_perm(0x64646464u, w, SEL0)) + off0;
    out[1] = as_f16x2(__builtin_amdgcn_perm(0x64646464u, w, SEL1)) + off1;
}
LQ_DEVICE f16x2 both(float v) { return f16x2{(_Float16)v, (_Float16)v}; }
LQ_DEVICE void int8_row(uint32_t w, f16x2 *out, f16x2 off = both(-1152.0f)) {
    int8_pairs<0x04010400u, 0x04030402u>(w, out, off, off);
}
LQ_DEVICE void int8_quad(uint32_t w, f16x2 *out, f16x2 off0 = both(-1152.0f), f16x2 off1 = both(-1152.0f)) {
    int8_pairs<0x04020400u, 0x04030401u>(w, out, off0, off1);
}
// `magic` is the fp16 pair (1024, 1024) in a vector register, so that mask and
// merge are one v_and_or_b32
LQ_DEVICE f16x2 int4_low(uint32_t w, uint32_t magic, f16x2 off = both(-1032.0f)) {
    return as_f16x2((w & 0x000F000Fu) | magic) + off;
}
LQ_DEVICE f16x2 int4_high(uint32_t w, uint32_t magic, f16x2 off = both(-72.0f)) {
    return __builtin_elementwise_fma(as_f16x2((w & 0x00F000F0u) | magic), both(0.0625f), off);
}
LQ_DEVICE uint32_t fp16_magic() {
    uint32_t m = 0x64006400u;
    asm volatile("" : "+v"(m));
    return m;
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
LQ_DEVICE float row_max(float v) {  // over 16 lanes
    v = fmaxf(v, dpp_f32<kDppXor1>(v));
    v = fmaxf(v, dpp_f32<kDppXor2>(v));
    v = fmaxf(v, dpp_f32<kDppHalfMirror>(v));
    return fmaxf(v, dpp_f32<kDppMirror>(v));
}
LQ_DEVICE float add_halves32(float v) { return swap_add32(v, v); }
LQ_DEVICE float add_halves16(float v) { return swap_add16(v, v); }
LQ_DEVICE float max4(f32x4 v) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); }

// A row without keys has the sum 0: zeros, and -inf for the log; a NaN goes on.
LQ_DEVICE float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
LQ_DEVICE float log_sum(float m, float l) { return l == 0.0f ? -__builtin_inff() : m * kLn2 + logf(l); }

// the power of two at or below a positive normal float
LQ_DEVICE float pow2_floor(float v) { return __uint_as_float(__float_as_uint(v) & 0x7F800000u); }

// ---- sharing out the work ----
//
// A unit is one tile of query rows of a sequence; its work is the sequence's
// keys in steps of STEP. All units' steps, one after another, are cut into
// equal spans, one for each of `cap` blocks of a key head, so every block has
// the same share whatever the lengths; lengths are read on the device, and the
// host needs to know no more than bounds. A block walks the pieces of units
// in its span: whole units are written out, a unit's part (the span's first or
// last piece) goes to the workspace and attn_join_kernel joins the parts.
struct Span {
    float *o;   // [2 cap][heads][rows of a tile][D], relative to the part's maximum
    float *ml;  // [2 cap][heads][rows of a tile][2]: maximum (log2) and sum
    int cap;
    int by_unit;           // every unit counts as one step: blocks take whole units
    uint32_t least, most;  // sequences of another number of query rows (all heads of a group) are not looked at
};

struct Piece {
    int64_t seq;
    int64_t start;  // the unit's first step among all steps
    int steps;      // steps of the unit
    uint32_t tile;  // the unit's tile in its sequence
    KvRows rows;
};

// One wave's view of all units: a lane a sequence, 64 at a time; the first 64
// are kept. Every piece is looked up from the first sequence on, which is little
// beside a decode batch of 512 sequences (100 tokens each, 8 heads: 79 us) and
// most of the time of one of 4096 (2135 us).
template <int STEP>
struct Schedule {
    struct Lane {
        KvRows rows;
        int steps;         // of each of the sequence's units
        int64_t all, upto;  // of all of them, and of the sequences up to this one
    };
    const KvBatch &bt;
    const Span &span;
    const int shift, group, row_tile, lane;
    Lane first;

    LQ_DEVICE Lane load(int64_t seq, int64_t before) const {
        Lane x{};
        x.steps = 1;
        if (seq < bt.b) {
            x.rows = kv_rows(bt, seq, shift);
            const uint32_t all_rows = (uint32_t)x.rows.n * (uint32_t)group;
            if (all_rows >= span.least && all_rows <= span.most) {
                int64_t keys = x.rows.first + x.rows.n < x.rows.len ? x.rows.first + x.rows.n : x.rows.len;
                keys = keys < 1 ? 1 : keys;  // a unit without keys is still written
                x.steps = span.by_unit ? 1 : (int)((keys + STEP - 1) / STEP);
                x.all = (int64_t)((all_rows + row_tile - 1) / (uint32_t)row_tile) * x.steps;
            }
        }
        x.upto = before + scan64(x.all);
        return x;
    }
    LQ_DEVICE Schedule(const KvBatch &b, const Span &sp, int sh, int g, int rt, int l)
        : bt(b), span(sp), shift(sh), group(g), row_tile(rt), lane(l) {
        first = load(lane, 0);
    }
    LQ_DEVICE int64_t total() const {
        int64_t sum = readlane64(first.upto, 63);
        for (int64_t s0 = 64; s0 < bt.b; s0 += 64) sum = readlane64(load(s0 + lane, sum).upto, 63);
        return sum;
    }
    // the unit that holds step pos (below the total)
    LQ_DEVICE Piece at(int64_t pos) const {
        Lane x = first;
        for (int64_t s0 = 0;;) {
            const uint64_t past = __ballot(x.upto > pos);
            if (past) {
                const int src = __ffsll((unsigned long long)past) - 1;
                Piece p;
                p.seq = s0 + src;
                p.steps = __builtin_amdgcn_readlane(x.steps, src);
                const int64_t start = readlane64(x.upto - x.all, src);
                const uint32_t j = (uint32_t)uniform_div(pos - start, p.steps);
                p.start = start + (int64_t)j * p.steps;
                // Early rows see fewer keys. Spans: tiles from both ends in turn,
                // so that neighbouring units together have about the same to do.
                // Whole units: the largest first, so that the last to start are
                // short (a prompt of 4096, 501 us in turn, 398 so).
                const uint32_t tiles = (uint32_t)uniform_div(readlane64(x.all, src), p.steps);
                p.tile = span.by_unit ? tiles - 1 - j : j & 1 ? tiles - 1 - (j >> 1) : j >> 1;
                p.rows.begin = readlane64(x.rows.begin, src);
                p.rows.n = readlane64(x.rows.n, src);
                p.rows.first = readlane64(x.rows.first, src);
                p.rows.len = readlane64(x.rows.len, src);
                return p;
            }
            const int64_t before = readlane64(x.upto, 63);
            s0 += 64;
            if (s0 >= bt.b) return Piece{0, pos, 1, 0, KvRows{0, 0, 0, 0}};  // not reached: pos is below the total
            x = load(s0 + lane, before);
        }
    }
};

// ---- few rows: one wave per run of 32 keys, no sharing between waves ----
//
// A tile's rows are the heads of the group, token by token. Wave w of a block
// walks a piece's 32-key tiles w, w + WAVES, ...; the next tile's keys are asked
// for as soon as this one's have been multiplied, its values after the second
// product, into the registers that just fell free. That leaves room for three
// waves a SIMD: a wave alone issues an instruction every 5-12 cycles, so the
// rate goes with the waves. The waves' results are joined in LDS.
//
// ROWS is 16, the width of the matrix instruction, or 8: then columns 0-7 and
// 8-15 hold the same rows, the first half of the lanes takes the softmax of
// the tile's first 16 keys and the second half that of the others (zeros
// elsewhere in p), and the two columns' outputs are added at the end. Half the
// scores, exponentials and scales a lane: INT4 decode of 16 sequences (70B
// heads) is bound by instructions, not bytes (28 us; 22 for the loads alone).
// Long contexts are bound by HBM: INT8 of 64 sequences, 1.42 GB in 216 us.
template <int D, int BITS, bool SYM, int ROWS>
struct Few {
    static constexpr int HALVES = 16 / ROWS;
    static constexpr int US = 2 / HALVES;            // 16-key groups whose softmax a lane takes
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
        f32x4 sk[US], sv[US], zk[US], zv[US];
    };
    // waves a SIMD that the registers allow
    static constexpr int OCC = D <= 128 && ROWS == 8 ? 3 : 2;
};
constexpr int kNoKey = 0x7FFFFF00;

// NT: streaming loads. The few-row kernel reads each code once (decode of 64
// sequences, 1.42 GB: 247 us with the default policy, 221 us streaming); the
// many-row kernel's blocks read what others have brought to L2.
template <int N, bool NT>
LQ_DEVICE void load_words(uint32_t *dst, const uint8_t *p) {
    if constexpr (N == 4) {
        const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
        const u32x4 v = NT ? __builtin_nontemporal_load(q) : *q;
        dst[0] = v[0]; dst[1] = v[1]; dst[2] = v[2]; dst[3] = v[3];
    } else {
        const u32x2 *q = reinterpret_cast<const u32x2 *>(p);
        const u32x2 v = NT ? __builtin_nontemporal_load(q) : *q;
        dst[0] = v[0]; dst[1] = v[1];
    }
}
// The lane's query row in fp16, scaled by a power of two (the row's largest
// element to [2^14, 2^15)); the sign of the softmax's scale goes to q, so that
// larger products are larger scores. The row's other elements are in the lanes
// 32 (MANY) or 16, 32 and 48 away. Returns what a product is to be multiplied
// by to be a score in log2; qsum: the sum of this lane's elements.
template <int STEPS, int BITS, bool SYM, bool MANY>
LQ_DEVICE float q_to_fp16(const u32x4 *raw, float scale, f16x8 *qf, float &qsum) {
    // magnitudes of bf16 order as their bits do, two to a word
    u16x2 top2 = {0, 0};
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            top2 = __builtin_elementwise_max(top2, __builtin_bit_cast(u16x2, raw[s][j] & 0x7FFF7FFFu));
    float amax = max_halves32(__uint_as_float((uint32_t)(top2[0] > top2[1] ? top2[0] : top2[1]) << 16));
    if (!MANY) amax = max_halves16(amax);
    int sh = 141 - (int)(__float_as_uint(amax) >> 23);
    sh = sh < -100 ? -100 : sh > 100 ? 100 : sh;
    const float up = scale == 0.0f ? 0.0f : copysignf(__uint_as_float((uint32_t)(sh + 127) << 23), scale);
    const float unscale = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = bf16_lo(raw[s][j]) * up;
            f[2 * j + 1] = bf16_hi(raw[s][j]) * up;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // the order in which a word's codes come out: nibbles 0 4 1 5 2 6 3 7
            const int src = BITS == 8 ? e : (e >> 1) + 4 * (e & 1);
            qf[s][e] = (_Float16)f[src];
            if (!SYM) qsum += (float)qf[s][e];
        }
    }
    return scale == 0.0f ? 1.0f : fmaxf(fabsf(scale) * kLog2e * unscale, 1e-37f);
}

template <int D, int BITS, bool SYM, int ROWS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, (Few<D, BITS, SYM, ROWS>::OCC)) void attn_few_kernel(AttnArgs a, Span span) {
    using C = Few<D, BITS, SYM, ROWS>;
    constexpr int LDO = D + 4;
    constexpr int kStride = 32 * WAVES;  // keys from one of a wave's tiles to its next
    __shared__ float lds_o[WAVES][ROWS][LDO];
    __shared__ float lds_m[WAVES][ROWS], lds_l[WAVES][ROWS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int row = n % ROWS, half = n / ROWS;  // the lane's row, and which keys' softmax it takes
    const int h = blockIdx.x % a.c.heads;
    const int block = blockIdx.x / a.c.heads;
    const int group = a.q_heads / a.c.heads;
    const int shift = a.c.page_shift, ps_mask = (1 << shift) - 1;
    const int pages = (int)a.c.pages;
    // byte offsets of this lane inside 16 keys' codes, and of its four keys' scales
    const uint32_t k_off = n * C::kRow + g * (C::VEC * 4), v_off = 4 * g * C::kRow + n * (C::VEC * 4);
    const uint32_t m_off = 4 * g;

    const uint32_t magic = fp16_magic();

    const Schedule<kStride> sched(a.batch, span, shift, group, ROWS, lane);
    const int64_t all_steps = sched.total(), share = uniform_div(all_steps + span.cap - 1, span.cap);
    const int64_t begin = block * share, end = begin + share < all_steps ? begin + share : all_steps;
    for (int64_t pos = begin; pos < end;) {
        const Piece piece = sched.at(pos);
        const int64_t seq = piece.seq;
        const uint32_t tile = piece.tile;
        const int step0 = (int)(pos - piece.start);
        int step1 = end - piece.start < piece.steps ? (int)(end - piece.start) : piece.steps;
        const bool whole = step0 == 0 && step1 == piece.steps;
        const int64_t slot_of = ((int64_t)(2 * block + (pos > begin)) * a.c.heads + h) * ROWS;
        pos = piece.start + step1;
        const int32_t *const table = a.batch.table + seq * a.batch.max_pages;
        const KvRows &rows = piece.rows;
        const uint32_t total = (uint32_t)rows.n * (uint32_t)group;
        // this lane's query row
        const uint32_t rr = tile * ROWS + row;
        const bool live = rr < total;
        const uint32_t tok = live ? rr / (uint32_t)group : 0;
        const int qh = h * group + (int)(live ? rr - tok * (uint32_t)group : 0);
        const uint32_t last_row = (tile * ROWS + ROWS - 1 < total ? tile * ROWS + ROWS - 1 : total - 1) / (uint32_t)group;
        const int row_pos = live ? (int)(rows.first + tok) : -1;              // last position the row sees
        const int safe = (int)(rows.first + tile * ROWS / (uint32_t)group);     // every row sees up to here
        int64_t kend64 = rows.first + last_row + 1;
        kend64 = kend64 > rows.len ? rows.len : kend64;
        const int kend = kend64 < 0 ? 0 : (int)kend64;
        if (span.by_unit) step1 = (kend + kStride - 1) / kStride;
        const int kbeg = step0 * kStride < kend ? step0 * kStride : kend;
        const int kstop = (int64_t)step1 * kStride < kend ? step1 * kStride : kend;
        const int top = (kstop - 1) & ~15;  // the piece's last 16 keys

        // pages of this lane's iteration of the wave, 64 iterations at a time
        int pid0 = 0, pid1 = 0;
        auto load_pages = [&](int it) {
            int k0 = kbeg + 32 * wave + kStride * (it + lane), k1 = k0 + 16;
            k0 = k0 < top ? k0 : top;
            k1 = k1 < top ? k1 : top;
            pid0 = table[k0 >> shift];
            pid1 = table[k1 >> shift];
        };
        // the page numbers are waited for here, so that reading one later does
        // not wait for the loads of codes issued since
        auto settle_pages = [&]() { asm volatile("" : "+v"(pid0), "+v"(pid1)); };
        // slots of a tile's two groups of 16 keys, and their first keys (kNoKey for
        // a page outside the pool)
        auto slots_of = [&](int it, int64_t *slots, int *keys) {
            const int key0 = kbeg + 32 * wave + kStride * it;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                int page = __builtin_amdgcn_readlane(u ? pid1 : pid0, it & 63);
                const int key = key0 + 16 * u;
                const bool in = (uint32_t)page < (uint32_t)pages;
                keys[u] = in ? key : kNoKey;
                page = in ? page : 0;
                const int kc = key < top ? key : top;
                slots[u] = (((int64_t)page * a.c.heads + h) << shift) + (kc & ps_mask);
            }
        };
        auto load_keys = [&](typename C::Tile &x, const int64_t *slots) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t *kp = a.c.k_codes + slots[u] * C::kRow;
#pragma unroll
                for (int j = 0; j < C::NV; ++j) load_words<C::VEC, true>(x.k[u] + j * C::VEC, kp + j * 64 + k_off);
            }
#pragma unroll
            for (int u = 0; u < C::US; ++u) {
                const int64_t at = (C::HALVES == 2 ? (half ? slots[1] : slots[0]) : slots[u]) + m_off;
                x.sk[u] = *reinterpret_cast<const f32x4 *>(a.c.k_scales + at);
                if (!SYM) x.zk[u] = *reinterpret_cast<const f32x4 *>(a.c.k_zeros + at);
            }
        };
        auto load_values = [&](typename C::Tile &x, const int64_t *slots) {
#pragma unroll
            for (int u = 0; u < C::US; ++u) {
                const int64_t at = (C::HALVES == 2 ? (half ? slots[1] : slots[0]) : slots[u]) + m_off;
                x.sv[u] = *reinterpret_cast<const f32x4 *>(a.c.v_scales + at);
                if (!SYM) x.zv[u] = *reinterpret_cast<const f32x4 *>(a.c.v_zeros + at);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t *vp = a.c.v_codes + slots[u] * C::kRow;
#pragma unroll
                for (int j = 0; j < C::NV; ++j) load_words<C::VEC, true>(x.v[u] + j * C::VEC, vp + j * 256 + v_off);
            }
        };
        const int first_key = kbeg + 32 * wave;
        const int its = kstop > first_key ? (kstop - first_key + kStride - 1) / kStride : 0;
        typename C::Tile x;
        int64_t slots[2] = {0, 0};
        int keys[2] = {0, 0};
        if (its > 0) load_pages(0);

        f16x8 qf[C::STEPS];
        float c1, qsum = 0.0f;
        {
            u32x4 raw[C::STEPS];
            const uint16_t *qp = a.q + (rows.begin + tok) * a.q_stride + (int64_t)qh * D;
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s) {
                constexpr int SPV = C::CPV / 8;
                const int d0 = C::CPV * (4 * (s / SPV) + g) + 8 * (s % SPV);
                raw[s] = live ? *reinterpret_cast<const u32x4 *>(qp + d0) : u32x4{0u, 0u, 0u, 0u};
            }
            settle_pages();
            if (its > 0) {  // in flight while q is made ready
                slots_of(0, slots, keys);
                load_keys(x, slots);
                load_values(x, slots);
            }
            c1 = q_to_fp16<C::STEPS, BITS, SYM, false>(raw, a.scale, qf, qsum);
            if (!SYM) qsum = add_halves16(add_halves32(qsum));
        }

        f32x4 o[C::TILES];
#pragma unroll
        for (int t = 0; t < C::TILES; ++t) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // m: reference of the row's scores (log2); sref: that of the value
        // scales, a power of two. Weights are exp2(score - m) kHead / sref (l
        // sums these), and times the value scale as the product's operand.
        float m = -1e30f, l = 0.0f, vz = 0.0f, sref = 0.0f, mm = -1e30f;

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
                    t[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(kf), qf[s], t[u], 0, 0, 0);
                }
            }
            int key_of[C::US];
            if constexpr (C::HALVES == 2) {
                key_of[0] = (half ? keys[1] : keys[0]) + 4 * g;
#pragma unroll
                for (int i = 0; i < 4; ++i) t[0][i] = half ? t[1][i] : t[0][i];
            } else {
                key_of[0] = keys[0] + 4 * g;
                key_of[C::US - 1] = keys[1] + 4 * g;
            }
            float tm = -__builtin_inff();
            int smi = 0;  // positive floats order as their bits do
#pragma unroll
            for (int u = 0; u < C::US; ++u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!SYM) t[u][i] = __builtin_fmaf(C::kMid - x.zk[u][i], qsum, t[u][i]);
                    t[u][i] *= x.sk[u][i];
                }
            }
            const bool masked = keys[0] + 15 > safe || keys[1] + 15 > safe || keys[1] + 15 >= kstop;
            const bool more = it + 1 < its;
            if (more) {
                if (((it + 1) & 63) == 0) {
                    load_pages(it + 1);
                    settle_pages();
                }
                slots_of(it + 1, slots, keys);
                load_keys(x, slots);
            }
            if (masked) {
                // keys some row does not see, or nobody: they may hold anything
#pragma unroll
                for (int u = 0; u < C::US; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key_of[u] + i;
                        if (key > row_pos || key >= kstop) t[u][i] = -__builtin_inff();
                        if (key >= kstop) {
                            x.sv[u][i] = 0.0f;
                            if (!SYM) x.zv[u][i] = 0.0f;
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < C::US; ++u) {
                tm = fmaxf(tm, max4(t[u]));
#pragma unroll
                for (int i = 0; i < 4; ++i) smi = max(smi, __float_as_int(x.sv[u][i]));
            }
            tm *= c1;
            float sm = __int_as_float(smi);
            if (__any(tm > m + kSlack || sm > sref * kScaleSlack)) {
                tm = max_halves16(max_halves32(tm));
                if constexpr (C::HALVES == 2) tm = fmaxf(tm, dpp_f32<kDppRowRor8>(tm));
                sm = max_halves16(max_halves32(sm));
                if constexpr (C::HALVES == 2) sm = fmaxf(sm, dpp_f32<kDppRowRor8>(sm));
                const float mn = fmaxf(m, tm);
                const float sn = fmaxf(fmaxf(sref, kScaleMin), pow2_floor(sm));
                const float by = __builtin_amdgcn_exp2f(m - mn) * (sref / sn);  // 0 before the first keys
                l *= by;
                vz *= by;
#pragma unroll
                for (int q = 0; q < C::TILES; ++q) o[q] *= by;
                m = mn;
                sref = sn;
                mm = m + (__builtin_amdgcn_logf(sn) - kHeadLog2);
            }
            f16x2 pb[4];
#pragma unroll
            for (int u = 0; u < C::US; ++u) {
                float pv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t[u][i], c1, -mm));
                    l += p;
                    pv[i] = p * x.sv[u][i];
                }
                pb[2 * u] = f16x2{(_Float16)pv[0], (_Float16)pv[2]};
                pb[2 * u + 1] = f16x2{(_Float16)pv[1], (_Float16)pv[3]};
                if (!SYM) {
                    // The zero's share, from the same rounded weights; from the
                    // unrounded ones what of it lies outside the codes, as they may
                    // vanish in fp16 where a tiny scale goes with a large zero.
                    constexpr float levels = 2.0f * C::kMid - 1.0f;
                    const f32x4 zv = x.zv[u];
                    const float low = fminf(fminf(zv[0], zv[1]), fminf(zv[2], zv[3]));
                    if (__any(!(low >= 0.0f && max4(zv) <= levels))) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float near = fminf(fmaxf(zv[i], 0.0f), levels);
                            vz = __builtin_fmaf(pv[i], zv[i] - near, vz);
                            x.zv[u][i] = near;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        vz = __builtin_fmaf((float)pb[2 * u + (i & 1)][i >> 1], x.zv[u][i] - C::kMid, vz);
                }
            }
            if constexpr (C::HALVES == 2) {
                // first half: keys of the first 16 and zeros; second half the other way round
                const uint32_t p0 = __builtin_bit_cast(uint32_t, pb[0]), p1 = __builtin_bit_cast(uint32_t, pb[1]);
                pb[0] = as_f16x2(half ? 0u : p0);
                pb[1] = as_f16x2(half ? 0u : p1);
                pb[2] = as_f16x2(half ? p0 : 0u);
                pb[3] = as_f16x2(half ? p1 : 0u);
            }
            const f16x8 pf = join(pb);
#pragma unroll
            for (int w = 0; w < C::KW; ++w) {
                f16x2 vf[4];
                if constexpr (BITS == 8) {
                    int8_quad(x.v[0][w], vf);
                    int8_quad(x.v[1][w], vf + 2);
                    o[w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(vf), pf, o[w], 0, 0, 0);
                } else {
                    const uint32_t v0 = x.v[0][w], v1 = x.v[1][w], v08 = v0 >> 8, v18 = v1 >> 8;
                    vf[0] = int4_low(v0, magic); vf[1] = int4_low(v08, magic);
                    vf[2] = int4_low(v1, magic); vf[3] = int4_low(v18, magic);
                    o[2 * w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(vf), pf, o[2 * w], 0, 0, 0);
                    vf[0] = int4_high(v0, magic); vf[1] = int4_high(v08, magic);
                    vf[2] = int4_high(v1, magic); vf[3] = int4_high(v18, magic);
                    o[2 * w + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join(vf), pf, o[2 * w + 1], 0, 0, 0);
                }
            }
            if (more) load_values(x, slots);
        }
        l = add_halves16(add_halves32(l));
        if (!SYM) vz = add_halves16(add_halves32(vz));
        if constexpr (C::HALVES == 2) {
            l += dpp_f32<kDppRowRor8>(l);
            if (!SYM) vz += dpp_f32<kDppRowRor8>(vz);
#pragma unroll
            for (int q = 0; q < C::TILES; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[q][i] += dpp_f32<kDppRowRor8>(o[q][i]);
        }

        // join the waves
        if (g == 0 && half == 0) {
            lds_m[wave][row] = m;
            lds_l[wave][row] = l * (sref * (1.0f / kHead));
        }
        __syncthreads();
        float mall = lds_m[0][row];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) mall = fmaxf(mall, lds_m[w][row]);
        const float f = __builtin_amdgcn_exp2f(m - mall) * (sref * (1.0f / kHead));
        if (half == 0) {
#pragma unroll
            for (int j = 0; j < C::NV; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // elements of word t of load j in matrix row 4 g + i
                    constexpr int EPW = 8 / BITS;
                    float *dst = &lds_o[wave][row][((j * 16 + 4 * g + i) * C::VEC) * EPW];
#pragma unroll
                    for (int t = 0; t < C::VEC * EPW; ++t) dst[t] = (o[j * C::VEC * EPW + t][i] - vz) * f;
                }
        }
        __syncthreads();
        constexpr int kTeam = 64 * WAVES / ROWS;  // lanes a row
        const int r = threadIdx.x / kTeam, c = threadIdx.x % kTeam;
        const uint32_t wr = tile * ROWS + r;
        if (wr < total) {
            float mr = lds_m[0][r];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) mr = fmaxf(mr, lds_m[w][r]);
            float lr = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) lr += lds_l[w][r] * __builtin_amdgcn_exp2f(lds_m[w][r] - mr);
            const uint32_t wt = wr / (uint32_t)group;
            const int64_t at = (rows.begin + wt) * a.q_heads + h * group + (wr - wt * (uint32_t)group);
            const float norm = !whole ? 1.0f : inverse_sum(lr);
#pragma unroll
            for (int d = 4 * c; d < D; d += 4 * kTeam) {
                f32x4 v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < WAVES; ++w) v += *reinterpret_cast<const f32x4 *>(&lds_o[w][r][d]);
                v *= norm;
                if (!whole) {
                    *reinterpret_cast<f32x4 *>(span.o + (slot_of + r) * D + d) = v;
                } else {
                    const bf16x2_t b0{(__bf16)v[0], (__bf16)v[1]}, b1{(__bf16)v[2], (__bf16)v[3]};
                    *reinterpret_cast<u32x2 *>(a.out + at * D + d) =
                        u32x2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
                }
            }
            if (c == 0) {
                if (!whole) {
                    float *ml = span.ml + (slot_of + r) * 2;
                    ml[0] = lr == 0.0f ? -__builtin_inff() : mr;
                    ml[1] = lr;
                } else if (a.lse) {
                    a.lse[at] = log_sum(mr, lr);
                }
            }
        }
        __syncthreads();  // the next piece reuses the buffers
    }
}

// ---- many rows: 128 or 256 query rows share each key tile through LDS ----
//
// W waves of 32 rows. Each key tile's codes are loaded once by the block (ahead
// of their use), turned into fp16 once and laid out in LDS as the 32 x 32 x 16
// matrix instruction reads them, so the conversion costs a 32 W-th of an
// operation per row and code. Tiles of 128 rows leave room for two blocks a CU
// (one's softmax beside the other's products), tiles of 256 for one. Two waves
// a SIMD are what the registers allow, and a wave alone issues a vector
// instruction every 5-12 cycles: the products (16 instructions of 32 cycles for
// 32 keys of 32 rows) and the softmax (some 150) together are the bound, not
// either rate: 522 to 626 us on different cards for a 2048-token chunk over 8192
// (770 to 920 TFLOP/s).
template <int D, int BITS, bool SYM, int W>
struct Many {
    static constexpr int ROWS = 32 * W;
    static constexpr int KT = D == 64 ? 16 * W : 8 * W;  // keys of a tile
    static constexpr int RING = 3;                 // tiles in LDS: in use, next, being written
    static constexpr int kRow = D * BITS / 8;
    static constexpr int KB = kRow * KT / (64 * W);  // key code bytes a thread
    static constexpr int TPK = 64 * W / KT;        // threads a key
    static constexpr int TP = 64 * W / (KT / 8);   // threads a pair of value quads
    static constexpr int VW = kRow / TP;           // value words a thread and quad
    static constexpr int DW = VW * 8 / BITS;       // value elements a thread
    static constexpr int STEPS = D / 16;           // score MFMAs per 32 keys
    static constexpr int JT = D / 32;              // output tiles
    static constexpr int CHUNKS = D / 8;           // 16-byte chunks of a key's fp16 row
    static constexpr float kMid = (float)(1 << (BITS - 1));

    static constexpr int KC = KB / BITS;           // 8-code chunks a thread brings of a key
    // Keys lie chunk by chunk ([chunk][key][8 elements]), each chunk's run a
    // little longer than its keys so that the threads of one key write to
    // different banks; values [16 keys][half][position][8 keys], position p
    // holding element (p % TP) DW + p / TP. Reads are runs of 16 bytes a lane.
    static constexpr int KPAD = KT + (D == 64 ? 2 : 1);
    struct Buf {
        f16x8 k[CHUNKS * KPAD], v[KT / 8 * D];
        float meta[4][KT];   // key scales, value scales, what is left of key and value zeros
        float stat[4][KT / 16];  // [1]: the largest value scale of each 16 keys
        int flags[KT / 16];      // kBad, kWideK, kWideV of each 16 keys
        // asymmetric: what is added to a code in the mantissa of 1024 (and, INT4,
        // of 64) to take the zero off it: keys twice each, values by quads in the
        // order 0 2 1 3
        uint32_t koff[SYM ? 1 : BITS == 4 ? 2 : 1][SYM ? 1 : KT];
        alignas(8) _Float16 voff[SYM ? 1 : BITS == 4 ? 2 : 1][SYM ? 4 : KT];
    };
    // Key zeros between -1024 and 1024 and value zeros among the codes (all but
    // those of keys and values far from 0 for their range) are taken off the codes
    // exactly in the conversion to fp16, once for all rows; what is left of others
    // (meta's zeros) is taken off the sums, in branches that these flags choose.
    // Scores and weights thus cost the same with zeros as without (ragged chunks
    // of 64-wide heads, INT8: 95 us, against 112 with every zero taken off the
    // sums).
    enum { kBad = 1, kWideK = 2, kWideV = 4 };
    struct Off {
        f16x2 k[2], v[2][2][2];  // [low, high nibble]; values [quad][tokens 0 2, 1 3][nibble]
    };
    struct Load {
        uint32_t k[KB / 4], v0[VW], v1[VW];
        float meta;
        int bad, dead;
    };
};

template <int N>
LQ_DEVICE void load_any(uint32_t *dst, const uint8_t *p) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) load_words<4, false>(dst + i, p + 4 * i);
    } else if constexpr (N == 2) {
        load_words<2, false>(dst, p);
    } else {
        dst[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

template <int D, int BITS, bool SYM, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void attn_many_kernel(AttnArgs a, Span span) {
    using C = Many<D, BITS, SYM, W>;
    __shared__ typename C::Buf lds[C::RING];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, half = lane >> 5;
    const int h = blockIdx.x % a.c.heads;
    const int block = blockIdx.x / a.c.heads;
    const int group = a.q_heads / a.c.heads;
    const int shift = a.c.page_shift, ps_mask = (1 << shift) - 1;
    const int pages = (int)a.c.pages;
    const uint32_t magic = fp16_magic();
    // what this thread brings of a tile: all its keys are of one group of 16
    const int my_key = threadIdx.x / C::TPK, my_part = threadIdx.x % C::TPK;  // in the tile
    const int my_group = D == 64 ? wave : wave >> 1;
    const int my_pair = threadIdx.x / C::TP, my_t = threadIdx.x % C::TP;      // 16-key step and half, position
    const uint32_t k_off = (my_key & 15) * C::kRow + my_part * C::KB;
    const uint32_t v_off = (my_pair & 1) * 4 * C::kRow + my_t * C::VW * 4;    // its second quad is 2 quads on
    // lanes 0-15 bring the key scales, 16-31 the value scales, then the zeros
    const float *const meta_src = (lane < 16             ? a.c.k_scales
                                   : SYM || lane < 32    ? a.c.v_scales
                                   : lane < 48           ? a.c.k_zeros
                                                         : a.c.v_zeros) + (lane & 15);

    // looked up anew for each piece: its registers are wanted inside
    const auto schedule = [&]() { return Schedule<C::KT>(a.batch, span, shift, group, C::ROWS, lane); };
    int64_t begin, end;
    {
        const int64_t all_steps = schedule().total(), share = uniform_div(all_steps + span.cap - 1, span.cap);
        begin = block * share;
        end = begin + share < all_steps ? begin + share : all_steps;
    }
    for (int64_t pos = begin; pos < end;) {
        const Piece piece = schedule().at(pos);
        const KvRows &rows = piece.rows;
        int step0 = (int)(pos - piece.start);
        int step1 = end - piece.start < piece.steps ? (int)(end - piece.start) : piece.steps;
        const bool whole = step0 == 0 && step1 == piece.steps;
        const int64_t slot_of = ((int64_t)(2 * block + (pos > begin)) * a.c.heads + h) * C::ROWS;
        pos = piece.start + step1;
        const uint32_t tile = piece.tile;
        const int32_t *const table = a.batch.table + piece.seq * a.batch.max_pages;
        const uint32_t total = (uint32_t)rows.n * (uint32_t)group;

        // this lane's query row, and the wave's first and last
        const uint32_t wave_row = tile * C::ROWS + wave * 32, rr = wave_row + n;
        const bool live = rr < total;
        const uint32_t tok = live ? rr / (uint32_t)group : 0;
        const int qh = h * group + (int)(live ? rr - tok * (uint32_t)group : 0);
        const uint32_t block_last = (tile * C::ROWS + C::ROWS - 1 < total ? tile * C::ROWS + C::ROWS - 1 : total - 1) / (uint32_t)group;
        const int row_pos = live ? (int)(rows.first + tok) : -1;
        const int safe = (int)(rows.first + wave_row / (uint32_t)group);
        int64_t kend64 = rows.first + block_last + 1;
        kend64 = kend64 > rows.len ? rows.len : kend64;
        const int kend = kend64 < 0 ? 0 : (int)kend64;
        if (span.by_unit) step1 = (kend + C::KT - 1) / C::KT;
        const int kbeg = step0 * C::KT < kend ? step0 * C::KT : kend;
        const int kstop = (int64_t)step1 * C::KT < kend ? step1 * C::KT : kend;
        const int its = (kstop - kbeg + C::KT - 1) / C::KT;
        const int top = (kstop - 1) & ~15;

        // pages of 64 groups of 16 keys ahead, a lane each
        int pid = 0;
        auto load_pages = [&](int it) {
            int k0 = kbeg + C::KT * it + 16 * lane;
            k0 = k0 < top ? k0 : top;
            pid = table[k0 >> shift];
        };
        constexpr int kAhead = 64 * 16 / C::KT;  // tiles of one such read
        auto load = [&](typename C::Load &x, int it) {
            if (it % kAhead == 0 && it > 0) {
                load_pages(it);
                asm volatile("" : "+v"(pid));
            }
            const int key0 = kbeg + C::KT * it + 16 * my_group;
            int page = __builtin_amdgcn_readlane(pid, (it % kAhead) * (C::KT / 16) + my_group);
            x.bad = (uint32_t)page >= (uint32_t)pages;
            page = x.bad ? 0 : page;
            const int kc = key0 < top ? key0 : top;
            const int64_t slot = (((int64_t)page * a.c.heads + h) << shift) + (kc & ps_mask);
            load_any<C::KB / 4>(x.k, a.c.k_codes + slot * C::kRow + k_off);
            const uint8_t *vp = a.c.v_codes + slot * C::kRow;
            load_any<C::VW>(x.v0, vp + v_off);
            load_any<C::VW>(x.v1, vp + 8 * C::kRow + v_off);
            x.dead = x.bad | (key0 + (lane & 15) >= kstop);
            x.meta = meta_src[slot];
        };
        // one 16-byte write of the tile: i below KC a chunk of keys, then values
        auto store_part = [&](const typename C::Load &x, typename C::Buf &b, int i, const typename C::Off &off) {
            f16x2 f[4];
            if (i < C::KC) {
                if constexpr (BITS == 8) {
                    int8_row(x.k[(2 * i) % (C::KB / 4)], f, off.k[0]);
                    int8_row(x.k[(2 * i + 1) % (C::KB / 4)], f + 2, off.k[0]);
                } else {
                    const uint32_t w = x.k[i % (C::KB / 4)], w8 = w >> 8;
                    f[0] = int4_low(w, magic, off.k[0]); f[1] = int4_high(w, magic, off.k[1]);
                    f[2] = int4_low(w8, magic, off.k[0]); f[3] = int4_high(w8, magic, off.k[1]);
                }
                b.k[(my_part * C::KC + i) * C::KPAD + my_key] = join(f);
            } else {
                const int e = i - C::KC;  // which of the thread's elements
                if constexpr (BITS == 8) {
                    int8_quad(x.v0[e % C::VW], f, off.v[0][0][0], off.v[0][1][0]);
                    int8_quad(x.v1[e % C::VW], f + 2, off.v[1][0][0], off.v[1][1][0]);
                } else {
                    const uint32_t v0 = x.v0[(e >> 1) % C::VW], v1 = x.v1[(e >> 1) % C::VW];
                    if (e & 1) {
                        f[0] = int4_high(v0, magic, off.v[0][0][1]); f[1] = int4_high(v0 >> 8, magic, off.v[0][1][1]);
                        f[2] = int4_high(v1, magic, off.v[1][0][1]); f[3] = int4_high(v1 >> 8, magic, off.v[1][1][1]);
                    } else {
                        f[0] = int4_low(v0, magic, off.v[0][0][0]); f[1] = int4_low(v0 >> 8, magic, off.v[0][1][0]);
                        f[2] = int4_low(v1, magic, off.v[1][0][0]); f[3] = int4_low(v1 >> 8, magic, off.v[1][1][0]);
                    }
                }
                b.v[my_pair * D + my_t + e * C::TP] = join(f);
            }
        };
        constexpr int kParts = C::KC + C::DW;
        // scales and zeros of the wave's 16 keys; returns the offsets of this
        // thread's own keys, which the wave itself has just written
        auto store_meta = [&](const typename C::Load &x, typename C::Buf &b) {
            typename C::Off off;
            // slots that hold nothing count as zeros
            float meta = x.dead ? (lane < 32 ? 0.0f : C::kMid) : x.meta;
            int flags = x.bad ? C::kBad : 0;
            if constexpr (SYM) {
                off.k[0] = both(-1024.0f - C::kMid);
                off.k[1] = both(-64.0f - C::kMid);
#pragma unroll
                for (int i = 0; i < 8; ++i) off.v[i >> 2][(i >> 1) & 1][i & 1] = off.k[i & 1];
            } else if (lane >= 32) {
                const float near = lane < 48 ? fminf(fmaxf(rintf(meta), -1024.0f), 1024.0f)
                                             : fminf(fmaxf(rintf(meta), 0.0f), 2.0f * C::kMid - 1.0f);
                meta -= near;
                const f16x2 low = both(-1024.0f - near), high = both(-64.0f - near);
                const int key = 16 * my_group + (lane & 15), quad = (key & ~3) | ((key & 1) << 1) | ((key >> 1) & 1);
                if (lane < 48) {
                    b.koff[0][key] = __builtin_bit_cast(uint32_t, low);
                    if (BITS == 4) b.koff[BITS == 4][key] = __builtin_bit_cast(uint32_t, high);
                } else {
                    b.voff[0][quad] = low[0];
                    if (BITS == 4) b.voff[BITS == 4][quad] = high[0];
                }
            }
            b.meta[lane >> 4][16 * my_group + (lane & 15)] = meta;
            b.stat[lane >> 4][my_group] = row_max(meta);
            if constexpr (!SYM) {
                const uint64_t wide = __ballot(lane >= 32 && meta != 0.0f);
                flags |= ((wide >> 32) & 0xFFFFu ? C::kWideK : 0) | (wide >> 48 ? C::kWideV : 0);
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
                for (int i = 0; i < (BITS == 4 ? 2 : 1); ++i) {
                    off.k[i] = as_f16x2(b.koff[i][my_key]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const u32x2 w = *reinterpret_cast<const u32x2 *>(&b.voff[i][16 * my_group + 8 * u + 4 * (my_pair & 1)]);
                        off.v[u][0][i] = as_f16x2(w[0]);
                        off.v[u][1][i] = as_f16x2(w[1]);
                    }
                }
            }
            b.flags[my_group] = flags;
            return off;
        };
        auto store = [&](const typename C::Load &x, typename C::Buf &b) {
            const typename C::Off off = store_meta(x, b);
#pragma unroll
            for (int i = 0; i < kParts; ++i) store_part(x, b, i, off);
        };

        typename C::Load x;
        if (its > 0) load_pages(0);
        // q as in the other kernel: fp16, scaled by a power of two
        f16x8 qf[C::STEPS];
        float c1, qsum = 0.0f;
        {
            u32x4 raw[C::STEPS];
            const uint16_t *qp = a.q + (rows.begin + tok) * a.q_stride + (int64_t)qh * D + 8 * half;
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s)
                raw[s] = live ? *reinterpret_cast<const u32x4 *>(qp + 16 * s) : u32x4{0u, 0u, 0u, 0u};
            asm volatile("" : "+v"(pid));
            if (its > 0) load(x, 0);
            c1 = q_to_fp16<C::STEPS, BITS, SYM, true>(raw, a.scale, qf, qsum);
            if (!SYM) qsum = add_halves32(qsum);
        }
        if (its > 0) store(x, lds[0]);
        if (its > 0) {
            load(x, 1);
            store(x, lds[1]);
            load(x, 2);
        }
        lds_barrier();

        f32x16 o[C::JT];
#pragma unroll
        for (int j = 0; j < C::JT; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
        float m = -1e30f, l = 0.0f, vz = 0.0f, sref = 0.0f, mm = -1e30f;
        constexpr int KBLK = C::KT / 32;

        // keys of block kb as the matrix instruction's operand, half of the steps
        auto key_operands = [&](const typename C::Buf &b, int kb, int from, f16x8 *kr) {
#pragma unroll
            for (int s = from; s < from + C::STEPS / 2; ++s) kr[s] = b.k[(2 * s + half) * C::KPAD + kb * 32 + n];
        };
        // Scores t of block kb of tile b times the key scales, part `part` of
        // `parts`, and their maximum: register i of the lane is key
        // 8 (i / 4) + 4 half + i % 4 of row n.
        auto key_scales = [&](const typename C::Buf &b, int kb, f32x4 *sk) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sk[r] = *reinterpret_cast<const f32x4 *>(&b.meta[0][kb * 32 + 8 * r + 4 * half]);
        };
        auto scale_scores = [&](const f32x4 *sk, f32x16 &t, float top, int part, int parts) {
#pragma unroll
            for (int i = part * 16 / parts; i < (part + 1) * 16 / parts; ++i) t[i] *= sk[i / 4][i % 4];
#pragma unroll
            for (int i = part * 16 / parts; i < (part + 1) * 16 / parts; i += 2) top = fmaxf(fmaxf(top, t[i]), t[i + 1]);
            return top;
        };
        // Mask and reference of these scores, tm their maximum.
        auto settle = [&](const typename C::Buf &b, int kb, int key0, f32x16 &t, float tm) {
            const int flags0 = __builtin_amdgcn_readfirstlane(b.flags[2 * kb]);
            const int flags1 = __builtin_amdgcn_readfirstlane(b.flags[2 * kb + 1]);
            const int bad0 = flags0 & C::kBad, bad1 = flags1 & C::kBad;
            const int first = key0 + 32 * kb;
            const float sm = fmaxf(b.stat[1][2 * kb], b.stat[1][2 * kb + 1]);
            if (first + 31 > safe || first + 32 > kstop || ((flags0 | flags1) & (C::kBad | C::kWideK))) {
                if (!SYM) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int at = kb * 32 + 8 * (i / 4) + 4 * half + i % 4;
                        t[i] = __builtin_fmaf(-b.meta[2][at] * b.meta[0][at], qsum, t[i]);
                    }
                }
                const int last = (row_pos < kstop ? row_pos : kstop - 1) - first - 4 * half;
                const int last0 = bad0 ? -1 : last, last1 = bad1 ? -1 : last;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    t[i] = 8 * (i / 4) + i % 4 > (i < 8 ? last0 : last1) ? -__builtin_inff() : t[i];
                tm = t[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) tm = fmaxf(tm, t[i]);
            }
            tm *= c1;
            if (__any(tm > m + kSlack || sm > sref * kScaleSlack)) {
                tm = max_halves32(tm);
                const float mn = fmaxf(m, tm);
                const float sn = fmaxf(fmaxf(sref, kScaleMin), pow2_floor(sm));
                const float by = __builtin_amdgcn_exp2f(m - mn) * (sref / sn);  // 0 before the first keys
                l *= by;
                vz *= by;
#pragma unroll
                for (int j = 0; j < C::JT; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[j][i] *= by;
                m = mn;
                sref = sn;
                mm = m + (__builtin_amdgcn_logf(sn) - kHeadLog2);
            }
            if (!SYM && ((flags0 | flags1) & C::kWideV)) {
                // of the unrounded weights: they may vanish in fp16 where a tiny
                // scale goes with a large zero. Their reference is hidden from the
                // compiler, which otherwise finds them equal to weigh's and moves
                // all weights ahead of this branch, away from the products: 2048
                // over 8192 tokens, 64 / 8 heads of 128, INT8 587 us, not 571.
                float ref = mm;
                asm volatile("" : "+v"(ref));
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int at = kb * 32 + 8 * (i / 4) + 4 * half + i % 4;
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t[i], c1, -ref));
                    vz = __builtin_fmaf(p, b.meta[1][at] * b.meta[3][at], vz);
                }
            }
        };
        // value scales of a lane's keys of block kb
        auto value_scales = [&](const typename C::Buf &b, int kb, int s, f32x4 *sv) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
                sv[r] = *reinterpret_cast<const f32x4 *>(&b.meta[1][kb * 32 + 16 * s + 8 * r + 4 * half]);
        };
        // The weights of t (block kb of tile b), their product with the values,
        // the next block's scores u = keys kr . q, and (with_store) the tile x on
        // its way to LDS, with the independent work side by side: JT groups of the
        // first 16 keys' weights, each beside a score instruction; JT groups of the
        // others', each beside a score and a value instruction; then the other
        // value instructions beside the scaling of u (peak: its maximum) and the
        // conversion of x. All of it is one run of instructions without a branch
        // but for asymmetric tiles of 128- and 256-wide heads, where the zeros'
        // part of store_meta, on half the lanes, comes between the weights and
        // the last value instructions. The 2048-token chunk took 538 us so, 550
        // with the scaling and the sums of the weights after the run. (Holding the
        // compiler to this order with scheduling barriers, or raising the wave's
        // priority over it, changed nothing beyond noise.)
        auto weigh = [&](const typename C::Buf &b, int kb, const f32x16 &t, const typename C::Buf &bn, int kn, f16x8 *kr,
                         f32x4 *sv, f32x16 &u, float &peak, bool with_store, typename C::Buf &to) {
            constexpr int EG = 8 / C::JT;  // weights of a group
            key_operands(bn, kn, C::STEPS / 2, kr);
            f16x8 vr[C::JT], pf[2];
#pragma unroll
            for (int j = 0; j < C::JT; ++j) vr[j] = b.v[(kb * 4 + half) * D + 32 * j + n];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = 0.0f;
#pragma unroll
            for (int s = 0; s < 2; ++s) {  // 16 keys
                float pv[8], even = 0.0f;
#pragma unroll
                for (int g = 0; g < C::JT; ++g) {
                    u = __builtin_amdgcn_mfma_f32_32x32x16_f16(kr[s * C::JT + g], qf[s * C::JT + g], u, 0, 0, 0);
                    if (s == 1) o[g] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vr[g], pf[0], o[g], 0, 0, 0);
#pragma unroll
                    for (int i = g * EG; i < (g + 1) * EG; ++i) {
                        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t[8 * s + i], c1, -mm));
                        if (i % 2) l += even + p;
                        else even = p;
                        pv[i] = p * sv[i / 4][i % 4];
                    }
                    if (s == 1) vr[g] = b.v[(kb * 4 + 2 + half) * D + 32 * g + n];
                }
                f16x2 pb[4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    pb[2 * r] = f16x2{(_Float16)pv[4 * r], (_Float16)pv[4 * r + 2]};
                    pb[2 * r + 1] = f16x2{(_Float16)pv[4 * r + 1], (_Float16)pv[4 * r + 3]};
                }
                pf[s] = join(pb);
                if (s == 0) value_scales(b, kb, 1, sv);
            }
            // used here, or the compiler moves the sums behind the branch below
            asm volatile("" : "+v"(l));
            typename C::Off off;
            if (with_store) off = store_meta(x, to);
            f32x4 sk[4];
            key_scales(bn, kn, sk);
            peak = -__builtin_inff();
#pragma unroll
            for (int g = 0; g < C::JT; ++g) {
                o[g] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vr[g], pf[1], o[g], 0, 0, 0);
                peak = scale_scores(sk, u, peak, g, C::JT);
                if (with_store) {
#pragma unroll
                    for (int i = g * kParts / C::JT; i < (g + 1) * kParts / C::JT; ++i) store_part(x, to, i, off);
                }
            }
        };

        // One tile: its first block's products are in t already. While a block's
        // weights are formed the next block's products run (the next tile's first
        // at the end; past the last tile whatever LDS holds, not used), and the
        // tile after that goes to LDS. A slot is written one barrier after its
        // last reader has passed and read one barrier after it is written.
        int now = 0;  // ring slot of the tile in use
        float peak = 0.0f;
        auto step = [&](int it, f32x16 &t, f32x16 &u) {
            const typename C::Buf &b = lds[now], &next = lds[now + 1 < C::RING ? now + 1 : now + 1 - C::RING];
            const int key0 = kbeg + C::KT * it;
            typename C::Buf &to = lds[now + 2 < C::RING ? now + 2 : now + 2 - C::RING];
            f16x8 kr[C::STEPS];
            f32x4 sv[2];
#pragma unroll
            for (int kb = 0; kb < KBLK; ++kb) {
                const bool last = kb == KBLK - 1;
                f32x16 &cur = kb & 1 ? u : t, &then = kb & 1 ? t : u;
                key_operands(last ? next : b, last ? 0 : kb + 1, 0, kr);
                value_scales(b, kb, 0, sv);
                settle(b, kb, key0, cur, peak);
                weigh(b, kb, cur, last ? next : b, last ? 0 : kb + 1, kr, sv, then, peak, last, to);
            }
            if (it + 3 < its) load(x, it + 3);
            lds_barrier();
            now = now + 1 < C::RING ? now + 1 : 0;
        };
        if (wave_row >= total) {  // no rows of its own: it only brings its part of the tiles
            for (int it = 0; it < its; ++it) {
                store(x, lds[now + 2 < C::RING ? now + 2 : now + 2 - C::RING]);
                if (it + 3 < its) load(x, it + 3);
                lds_barrier();
                now = now + 1 < C::RING ? now + 1 : 0;
            }
        } else if (its > 0) {
            f32x16 ta, tb;
            f16x8 kr[C::STEPS];
            key_operands(lds[0], 0, 0, kr);
            key_operands(lds[0], 0, C::STEPS / 2, kr);
#pragma unroll
            for (int i = 0; i < 16; ++i) ta[i] = 0.0f;
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s) ta = __builtin_amdgcn_mfma_f32_32x32x16_f16(kr[s], qf[s], ta, 0, 0, 0);
            f32x4 sk[4];
            key_scales(lds[0], 0, sk);
            peak = scale_scores(sk, ta, -__builtin_inff(), 0, 1);
            for (int it = 0; it < its; ++it) {
                step(it, ta, tb);
                if constexpr (KBLK == 1) {
                    if (++it >= its) break;
                    step(it, tb, ta);
                }
            }
        }
        lds_barrier();  // nobody reads the ring any more when the next piece fills it
        l = add_halves32(l);
        if (!SYM) vz = add_halves32(vz);
        if (live) {
            const int64_t at = (rows.begin + tok) * a.q_heads + qh;
            const int64_t part = slot_of + wave * 32 + n;
            l *= sref * (1.0f / kHead);
            const float f = (whole ? inverse_sum(l) : 1.0f) * (sref * (1.0f / kHead));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int mrow = 8 * (i / 4) + 4 * half + i % 4;
#pragma unroll
                for (int g = 0; g < C::TP / 32; ++g) {
                    // output tiles j = g, g + TP / 32, ...: DW neighbouring elements
                    float v[C::DW];
#pragma unroll
                    for (int e = 0; e < C::DW; ++e) v[e] = (o[e * (C::TP / 32) + g][i] - vz) * f;
                    const int d = (g * 32 + mrow) * C::DW;
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < C::DW; e += 2)
                            *reinterpret_cast<float2 *>(span.o + part * D + d + e) = float2{v[e], v[e + 1]};
                    } else {
#pragma unroll
                        for (int e = 0; e < C::DW; e += 2) {
                            const bf16x2_t b{(__bf16)v[e], (__bf16)v[e + 1]};
                            *reinterpret_cast<uint32_t *>(a.out + at * D + d + e) = __builtin_bit_cast(uint32_t, b);
                        }
                    }
                }
            }
            if (half == 0) {
                if (!whole) {
                    span.ml[part * 2] = l == 0.0f ? -__builtin_inff() : m;
                    span.ml[part * 2 + 1] = l;
                } else if (a.lse) {
                    a.lse[at] = log_sum(m, l);
                }
            }
        }
    }
}

// Joins the parts of the units that were cut: one block for each border between
// two spans and key head, which takes the unit that lies across it if this is
// the unit's first border. D / 4 lanes a row, four parts' loads in flight.
template <int D, int ROWS, int STEP>
LQ_DEVICE void join_parts(const AttnArgs &a, const Span &span, int block, int part, int parts_of_rows) {
    constexpr int W = D / 4, kTeams = 256 / W;
    const int lane = threadIdx.x & 63;
    const int h = block % a.c.heads;
    const int64_t border = block / a.c.heads + 1;
    const int group = a.q_heads / a.c.heads;
    const Schedule<STEP> sched(a.batch, span, a.c.page_shift, group, ROWS, lane);
    const int64_t all_steps = sched.total(), share = uniform_div(all_steps + span.cap - 1, span.cap);
    if (border * share >= all_steps) return;
    const Piece p = sched.at(border * share);
    if (p.start == border * share || p.start < (border - 1) * share) return;  // not across, or an earlier border's
    const int64_t last = uniform_div(p.start + p.steps - 1, share);                 // the unit's last block
    const int parts = (int)(last - border) + 2;
    // the unit's first part is its block's first piece if it starts there
    const int64_t slot0 = 2 * (border - 1) + (p.start > (border - 1) * share), slot1 = 2 * border;
    const KvRows &rows = p.rows;
    const uint32_t total = (uint32_t)rows.n * (uint32_t)group;
    const int c = threadIdx.x % W;
    for (int r = part * kTeams + threadIdx.x / W; r < ROWS; r += kTeams * parts_of_rows) {
        const uint32_t wr = p.tile * ROWS + r;
        if (wr >= total) break;
        auto slot = [&](int i) { return ((i == 0 ? slot0 : slot1 + 2 * (i - 1)) * a.c.heads + h) * ROWS + r; };
        // maximum and sum: each lane takes some parts, then the lanes' join
        float m = -__builtin_inff(), l = 0.0f;
        for (int i = c; i < parts; i += W) {
            const float2 x = reinterpret_cast<const float2 *>(span.ml)[slot(i)];
            const float mn = fmaxf(m, x.x);
            if (mn > -__builtin_inff()) l = l * __builtin_amdgcn_exp2f(m - mn) + x.y * __builtin_amdgcn_exp2f(x.x - mn);
            m = mn;
        }
        const float mall = fmaxf(team_max<W>(m), -1e30f);
        l = team_sum<W>(l * __builtin_amdgcn_exp2f(m - mall));
        f32x4 v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const int64_t at = slot(i);
            v += *reinterpret_cast<const f32x4 *>(span.o + at * D + 4 * c) *
                 __builtin_amdgcn_exp2f(span.ml[2 * at] - mall);
        }
        v *= inverse_sum(l);
        const uint32_t wt = wr / (uint32_t)group;
        const int64_t at = (rows.begin + wt) * a.q_heads + h * group + (wr - wt * (uint32_t)group);
        const bf16x2_t b0{(__bf16)v[0], (__bf16)v[1]}, b1{(__bf16)v[2], (__bf16)v[3]};
        *reinterpret_cast<u32x2 *>(a.out + at * D + 4 * c) =
            u32x2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
        if (c == 0 && a.lse) a.lse[at] = log_sum(mall, l);
    }
}

constexpr int kJoinY = 8;  // blocks that share a unit of many rows
template <int D, int ROWS, int STEP>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Span span) {
    join_parts<D, ROWS, STEP>(a, span, blockIdx.x, blockIdx.y, gridDim.y);
}
// Both launches' parts at once: `many` borders and heads of tiles of ROWS rows
// (kJoinY blocks each), then those of 16-row tiles.
template <int D, int ROWS, int STEP, int FEWSTEP>
__global__ __launch_bounds__(256) void attn_join_both_kernel(AttnArgs a, Span span, Span few, int many) {
    const int i = blockIdx.x;
    if (i < many * kJoinY)
        join_parts<D, ROWS, STEP>(a, span, i / kJoinY, i % kJoinY, kJoinY);
    else
        join_parts<D, 16, FEWSTEP>(a, few, i - many * kJoinY, 0, 1);
}

// One launch of a kernel (and of the join): the sequences it takes, its tile's
// rows, blocks a key head and workspace.
struct Pass {
    int row_tile, cap, by_unit;
    uint32_t least, most;
    int64_t bytes;
};
struct Plan {
    Pass pass[2];
    int passes;
    int64_t bytes;
};
constexpr int kFewWaves = 4, kFewStep = 32 * kFewWaves;

Pass pass_of(int row_tile, int64_t rows, int64_t group, int64_t heads, int64_t head_dim, int bits, int64_t b, int64_t kv,
             int64_t n) {
    Pass p{};
    p.row_tile = row_tile;
    p.least = 1;
    p.most = 0xFFFFFFFFu;
    const int64_t units = (rows * group + row_tile - 1) / row_tile + b;  // at most
    const int64_t tiles = (n * group + row_tile - 1) / row_tile;         // of a sequence
    const int64_t step = row_tile < 128 ? kFewStep : row_tile / (head_dim == 64 ? 2 : 4);
    // What the kernels' registers allow on 256 CUs: all blocks run at once, and
    // more spans only repeat the fixed part (twice as many for many rows: 2 chunks
    // beside single tokens 146 us, not 128; 64-wide heads 111, not 95). Single
    // tokens' kernel (row_tile 8) has room for three blocks a CU. The third pays
    // where a token's codes are few bytes, as the instructions per byte bound it
    // then, and costs some of HBM's rate otherwise. 512 and 768 blocks, up to 8192
    // tokens: INT4 of 128-wide heads, 8 sequences 25.5 and 24.9 us, 16 35.7 and
    // 33.2, 64 89.4 and 83.0 (up to 16384 158 and 146); INT8 of 64-wide heads, 64
    // sequences 30.0 and 27.9; INT8 of 128-wide heads, 16 sequences 42.7 and 43.4,
    // 24 56.4 and 58.3, 64 124 and 125 (up to 16384 230 and 232).
    const int64_t unit_steps = (kv + step - 1) / step < 1 ? 1 : (kv + step - 1) / step;
    const int64_t likely = b * tiles < units ? b * tiles : units;
    const bool thin = head_dim <= 128 && head_dim * bits <= 512;  // up to 64 bytes
    const int64_t blocks = row_tile == 256 ? 256 : row_tile == 8 && thin ? 768 : 512;
    int64_t cap = (blocks + heads - 1) / heads;
    // Blocks take whole units, and nothing is joined.
    if (row_tile >= 128) {
        // Chunks: cutting units costs about what 1200 more keys of each block do
        // (parts written, read and joined, more first loads); whole units cost
        // the last round's idle blocks, and at least the longest unit's time.
        // Measured, 64 / 8 heads of 128, spans and units: prompts of 1100, 1800
        // and 3000 85 and 57, 125 and 97, 263 and 225 us; 2048 over 8192 581 and
        // 579; 1500 over 8192 (1.5 rounds) 484 and 519; 512 over 4096 107 and 139;
        // two prompts of 4000 703 and 631; four ragged chunks of up to 1000 over
        // up to 4000 349 and 381, of 700 over 3000 218 and 200 (spans are taken).
        // Lengths other than the longest are not known here: half of it on the
        // average, and short contexts before the rows only.
        constexpr int64_t kCut = 1200;
        const int64_t slots = row_tile == 256 || head_dim == 256 ? 256 : 512, load = likely * heads;
        const int64_t mean = b == 1 ? kv - (n < kv ? n : kv) / 2 : kv / 2, prior = n < kv ? kv - n : 0;
        const int64_t idle = (load + slots - 1) / slots * slots - load;
        p.by_unit = load >= 4 * slots || (kv <= load * mean / slots + kCut && (b == 1 ? idle * prior <= kCut * slots : prior <= kCut));
    } else {
        // Decode batches of short contexts, which would spend longer on the
        // second launch, and of up to 2048 tokens where units fill the card. Spans
        // and units, INT8 of 128-wide heads: 1 x 1003 tokens on one head 16.8 and
        // 12.2 us a pass, 64 x 500 on 8 heads 21.8 and 14.5; 4 x 2000 on 8 heads
        // 16.2 and 22.2, 16 x 2000 19.8 and 23.4, 32 x 2000 27.0 and 25.1, 64 x
        // 2000 41.3 and 39.7 (INT4 asymmetric: 16 18.2 and 24.1, 32 24.4 and 24.9,
        // 64 35.2 and 30.7).
        p.by_unit = kv <= 1024 || (kv <= 2048 && likely * heads >= 256);
    }
    if (p.by_unit) cap = likely;
    // no more blocks than steps of work
    if (cap > units * unit_steps) cap = units * unit_steps;
    if (cap * heads > (1 << 22)) cap = (1 << 22) / heads;  // blocks that walk on, within the launch limits
    p.cap = (int)cap;
    p.bytes = cap > 1 && !p.by_unit ? (2 * cap * heads * row_tile * (head_dim + 2) * 4 + 255) / 256 * 256 : 0;
    return p;
}

Plan plan_of(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int bits, int64_t b, int64_t room,
             int64_t max_rows, int64_t max_kv) {
    Plan p{};
    const int64_t n = max_rows <= 0 || max_rows > rows ? rows : max_rows;
    const int64_t kv = max_kv <= 0 || max_kv > room ? room : max_kv;
    const int64_t group = q_heads / heads;
    auto pass = [&](int row_tile) { return pass_of(row_tile, rows, group, heads, head_dim, bits, b, kv, n); };
    p.passes = 1;
    if (n * group <= 16) {
        p.pass[0] = pass(n * group <= 8 ? 8 : 16);
    } else {
        // Tiles of 256 rows where a sequence fills them on the average (a
        // 2048-token chunk of the 70B heads in tiles of 128: 620 us, of 256:
        // 539; ragged chunks of 64-wide heads 99 and 95), of 128 otherwise. In a
        // batch of single tokens beside few chunks (the others than the longest
        // have few rows) the sequences of up to 16 rows go to the kernel for few
        // rows in a launch of their own (10 single tokens beside 2 chunks: 128
        // us, 160 in one); one launch joins both kinds' parts (133 with two).
        p.pass[0] = pass(rows * group >= 256 * b && head_dim != 256 ? 256 : 128);
        // That launch is sized by what such sequences can hold, one tile each: at
        // most b units, however many rows the chunks have (39 beside a chunk of
        // 300 on one head, 1500 tokens: 49.7 us, 60.6 by the chunk's rows).
        if (b >= 4 && group <= 16 && (rows - n) * group <= 64 * (b - 1)) {
            p.pass[0].least = 17;
            p.pass[1] = pass_of(16, 0, group, heads, head_dim, bits, b, kv, 1);
            p.pass[1].most = 16;
            p.passes = 2;
        }
    }
    p.bytes = p.pass[0].bytes + p.pass[1].bytes;
    return p;
}

}  // namespace

int64_t attention_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t b,
                                  int64_t max_pages, int64_t page_size, int64_t max_rows, int64_t max_kv) {
    // of either format: INT4's blocks are as many as INT8's or more
    return plan_of(rows, q_heads, heads, head_dim, 4, b, max_pages * page_size, max_rows, max_kv).bytes;
}

static Span span_of(const AttnArgs &a, const Pass &p, char *workspace) {
    float *o = reinterpret_cast<float *>(workspace);
    return {o, o + (int64_t)2 * p.cap * a.c.heads * p.row_tile * a.c.head_dim, p.cap, p.by_unit, p.least, p.most};
}
static uint32_t borders_of(const AttnArgs &a, const Pass &p) {  // and key heads: blocks of the join
    return p.by_unit ? 0 : (uint32_t)((p.cap - 1) * a.c.heads);
}

template <int D, int BITS, bool SYM, int ROWS>
static hipError_t launch_tiles(const AttnArgs &a, const Pass &p, const Span &span, hipStream_t st) {
    const dim3 grid((uint32_t)(p.cap * a.c.heads));
    if constexpr (ROWS < 128)
        hipLaunchKernelGGL((attn_few_kernel<D, BITS, SYM, ROWS, kFewWaves>), grid, dim3(64 * kFewWaves), 0, st, a, span);
    else
        hipLaunchKernelGGL((attn_many_kernel<D, BITS, SYM, ROWS / 32>), grid, dim3(2 * ROWS), 0, st, a, span);
    return hipGetLastError();
}

// The pass's kernel and the join; with `few`, the kernel for few rows between
// them (its workspace behind the pass's own) and one join for both.
template <int D, int BITS, bool SYM, int ROWS>
static hipError_t launch_pass(const AttnArgs &a, const Pass &p, const Pass *few, hipStream_t st) {
    char *ws = static_cast<char *>(a.workspace);
    const Span span = span_of(a, p, ws);
    hipError_t e = launch_tiles<D, BITS, SYM, ROWS>(a, p, span, st);
    if (e != hipSuccess) return e;
    const uint32_t borders = borders_of(a, p);
    constexpr int step = ROWS < 128 ? kFewStep : Many<D, BITS, SYM, (ROWS < 128 ? 128 : ROWS) / 32>::KT;
    if constexpr (ROWS >= 128) {
        if (few) {
            const Span small = span_of(a, *few, ws + p.bytes);
            e = launch_tiles<D, BITS, SYM, 16>(a, *few, small, st);
            const uint32_t blocks = borders * kJoinY + borders_of(a, *few);
            if (e != hipSuccess || blocks == 0) return e;
            hipLaunchKernelGGL((attn_join_both_kernel<D, ROWS, step, kFewStep>), dim3(blocks), dim3(256), 0, st, a, span,
                               small, (int)borders);
            return hipGetLastError();
        }
    }
    if (borders == 0) return e;
    hipLaunchKernelGGL((attn_join_kernel<D, ROWS, step>), dim3(borders, ROWS < 128 ? 1 : kJoinY), dim3(256), 0, st, a, span);
    return hipGetLastError();
}

template <int D, int BITS, bool SYM>
static hipError_t launch_plan(const AttnArgs &a, const Plan &p, hipStream_t st) {
    const Pass *few = p.passes == 2 ? &p.pass[1] : nullptr;
    switch (p.pass[0].row_tile) {
        case 8: return launch_pass<D, BITS, SYM, 8>(a, p.pass[0], nullptr, st);
        case 16: return launch_pass<D, BITS, SYM, 16>(a, p.pass[0], nullptr, st);
        case 128: return launch_pass<D, BITS, SYM, 128>(a, p.pass[0], few, st);
        default: return launch_pass<D, BITS, SYM, D == 256 ? 128 : 256>(a, p.pass[0], few, st);
    }
}

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st) {
    const Plan p = plan_of(a.batch.rows, a.q_heads, a.c.heads, a.c.head_dim, a.c.bits, a.batch.b,
                           a.batch.max_pages << a.c.page_shift, a.max_rows, a.max_kv);
#define LQ_ATTN(D, BITS, SYM) \
    if (a.c.head_dim == D && a.c.bits == BITS && (a.c.symmetric != 0) == SYM) return launch_plan<D, BITS, SYM>(a, p, st);
#define LQ_ATTN_D(D) LQ_ATTN(D, 4, false) LQ_ATTN(D, 4, true) LQ_ATTN(D, 8, false) LQ_ATTN(D, 8, true)
    LQ_ATTN_D(64) LQ_ATTN_D(128) LQ_ATTN_D(256)
#undef LQ_ATTN_D
#undef LQ_ATTN
    return hipErrorInvalidValue;
}

}  // namespace lq
