// codes.hpp -- cached codes and query rows as operands of the fp16 matrix
// instructions, for the kernels that multiply them.
#pragma once
#include "common.hpp"

namespace lq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896341f;

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
LQ_DEVICE float add_halves32(float v) { return swap_add32(v, v); }
LQ_DEVICE float add_halves16(float v) { return swap_add16(v, v); }

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

}  // namespace lq
