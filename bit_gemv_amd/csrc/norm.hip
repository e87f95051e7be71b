// norm.hip -- residual addition, root-mean-square norm and per-token INT8 in
// one kernel (rms_norm_int8).
//
// Per row: h = x + residual, r = (sum h^2 / k + eps)^-1/2, y = (h r) w,
// s = max|y| / 127, q = round(y / s). The row is read once and stays in
// registers over both reductions; the kernel is bound by HBM (2-4 bytes of x,
// 2 x 2 of a bf16 residual and 1 of codes per element; 8192 rows of 8192 from
// fp32 107 us, 5.6 TB/s), a few rows by latency (one row 4.4 us). The sum of squares is
// in fp64: products of fp32 values are exact there and a sum of k terms errs by
// at most k 2^-53 of itself, so after its one rounding to fp32 r is the definition's
// value unless that lies within 2^-39 (k = 8192) of the middle between two floats;
// only there could another order of the sum give another last bit.
#include "common.hpp"
#include "launch.hpp"

namespace lq {

namespace {

// 8 consecutive elements as fp32, from bf16 (one 16-byte load) or fp32 (two)
template <bool F32>
struct Raw8 {
    u32x4 a;
};
template <>
struct Raw8<true> {
    u32x4 a, b;
};

template <bool F32>
LQ_DEVICE Raw8<F32> load8(const void *p, int64_t e) {
    if constexpr (F32) {
        const u32x4 *q = reinterpret_cast<const u32x4 *>(static_cast<const float *>(p) + e);
        return {q[0], q[1]};
    } else {
        return {*reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + e)};
    }
}

template <bool F32>
LQ_DEVICE void widen8(const Raw8<F32> &r, float *f) {
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = __uint_as_float(r.a[j]);
            f[4 + j] = __uint_as_float(r.b[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = bf16_lo(r.a[j]);
            f[2 * j + 1] = bf16_hi(r.a[j]);
        }
    }
}

template <bool F32>
LQ_DEVICE void store8(void *p, int64_t e, const float *f) {
    if constexpr (F32) {
        f32x4 *q = reinterpret_cast<f32x4 *>(static_cast<float *>(p) + e);
        q[0] = f32x4{f[0], f[1], f[2], f[3]};
        q[1] = f32x4{f[4], f[5], f[6], f[7]};
    } else {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x2_t b{(__bf16)f[2 * j], (__bf16)f[2 * j + 1]};
            v[j] = __builtin_bit_cast(uint32_t, b);
        }
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + e) = v;
    }
}

enum { kNoRes = 0, kResBf16 = 1, kResF32 = 2 };

// h of 8 elements of each of the lane's NL pieces of one chunk; zeros past k.
// All loads are issued before any arithmetic.
template <int TPB, int NL, bool XF32, int RES>
LQ_DEVICE void load_h(const void *x, const void *res, int64_t row0, int64_t k, int64_t c0, int t, float h[NL][8]) {
    constexpr bool RF32 = RES == kResF32;
    Raw8<XF32> xv[NL];
    Raw8<RF32> rv[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int64_t e = c0 + (int64_t)(i * TPB + t) * 8;
        if (e < k) {
            xv[i] = load8<XF32>(x, row0 + e);
            if (RES != kNoRes) rv[i] = load8<RF32>(res, row0 + e);
        } else {
            xv[i] = Raw8<XF32>{};
            rv[i] = Raw8<RF32>{};
        }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        widen8<XF32>(xv[i], h[i]);
        if (RES != kNoRes) {
            float r[8];
            widen8<RF32>(rv[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        }
    }
}

// One block of TPB lanes per row, in chunks of NL * TPB * 8 elements. ONE:
// the row is one chunk, read once and kept; otherwise it is read once per
// reduction and once more for the codes, and residual_out (which may be
// residual) is written in that last pass only.
template <int TPB, int NL, bool XF32, int RES, bool ONE>
__global__ __launch_bounds__(TPB) void rms_norm_int8_kernel(const void *x, const void *res, const void *__restrict__ w,
                                                             int w_f32, int64_t k, double eps, void *res_out,
                                                             int8_t *__restrict__ qx, float *__restrict__ sx) {
    constexpr int kWaves = TPB / 64;
    constexpr int64_t kChunk = (int64_t)NL * TPB * 8;
    __shared__ double red_sum[kWaves];
    __shared__ float red_max[kWaves];
    const int64_t row0 = (int64_t)blockIdx.x * k;
    const int t = threadIdx.x;
    const int64_t nch = ONE ? 1 : (k + kChunk - 1) / kChunk;
    float h[NL][8];

    double ss = 0.0;
    for (int64_t ch = 0; ch < nch; ++ch) {
        load_h<TPB, NL, XF32, RES>(x, res, row0, k, ch * kChunk, t, h);
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)h[i][j], (double)h[i][j], ss);
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) ss += __shfl_xor(ss, m, 64);
    if ((t & 63) == 0) red_sum[t >> 6] = ss;
    __syncthreads();
    ss = red_sum[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) ss += red_sum[i];
    // with eps 0 a row of zeros, or of rms below 2^-128, has no fp32 r: the largest
    // float stands for it, so that zeros stay zeros and nothing becomes NaN
    float r = (float)(1.0 / sqrt(ss / (double)k + eps));
    r = r > 3.402823466e+38f ? 3.402823466e+38f : r;

    // y in place of h
    auto scale_h = [&](int64_t c0) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int64_t e = c0 + (int64_t)(i * TPB + t) * 8;
            float wf[8] = {};
            if (e < k) {
                if (w_f32)
                    widen8<true>(load8<true>(w, e), wf);
                else
                    widen8<false>(load8<false>(w, e), wf);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = (h[i][j] * r) * wf[j];
        }
    };
    auto store_h = [&](int64_t c0) {
        if (RES == kNoRes || !res_out) return;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int64_t e = c0 + (int64_t)(i * TPB + t) * 8;
            if (e < k) store8<RES == kResF32>(res_out, row0 + e, h[i]);
        }
    };

    float a = 0.0f;
    for (int64_t ch = 0; ch < nch; ++ch) {
        if (!ONE) load_h<TPB, NL, XF32, RES>(x, res, row0, k, ch * kChunk, t, h);
        if (ONE) store_h(0);
        scale_h(ch * kChunk);
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(h[i][j]));
    }
    a = team_max<64>(a);
    if ((t & 63) == 0) red_max[t >> 6] = a;
    __syncthreads();
    a = red_max[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) a = fmaxf(a, red_max[i]);
    const float am = a < kFloor ? kFloor : a;
    const float s = am / 127.0f;
    // y / s through div_rn with RN(1 / s): the IEEE quotient here, since
    // |y| <= am = 127 s, s >= 1e-8 / 127 and 1 / s are normal, and a quotient
    // of magnitude 1/2 or more has normal residuals (smaller ones round to 0)
    const float inv = 1.0f / s;
    for (int64_t ch = 0; ch < nch; ++ch) {
        if (!ONE) {
            load_h<TPB, NL, XF32, RES>(x, res, row0, k, ch * kChunk, t, h);
            store_h(ch * kChunk);
            scale_h(ch * kChunk);
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int64_t e = ch * kChunk + (int64_t)(i * TPB + t) * 8;
            if (e >= k) continue;
            // |RN(y / s)| <= 127 (1 + 2^-23) rounds to at most 127, so no
            // clamp; adding 2^23 + 256 rounds to an integer (ties to even)
            // whose low byte is the two's-complement code
            uint32_t c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = __float_as_uint(div_rn(h[i][j], s, inv) + 8388864.0f);
            const uint32_t lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u),
                                                      __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), 0x05040100u);
            const uint32_t hi = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[7], c[6], 0x0C0C0400u),
                                                      __builtin_amdgcn_perm(c[5], c[4], 0x0C0C0400u), 0x05040100u);
            *reinterpret_cast<u32x2 *>(qx + row0 + e) = u32x2{lo, hi};
        }
    }
    if (t == 0) sx[blockIdx.x] = s;
}

// a.t at most 2^21: a launch's lanes in one dimension stay below 2^32
template <int TPB, int NL, bool ONE>
hipError_t launch_shape(const NormArgs &a, hipStream_t st) {
    const int res = !a.residual ? kNoRes : a.residual_f32 ? kResF32 : kResBf16;
#define LQ_NORM(XF32, RES)                                                                                        \
    if ((a.x_f32 != 0) == XF32 && res == RES) {                                                                   \
        hipLaunchKernelGGL((rms_norm_int8_kernel<TPB, NL, XF32, RES, ONE>), dim3((uint32_t)a.t), dim3(TPB), 0, st, \
                           a.x, a.residual, a.weight, a.weight_f32, a.k, a.eps, a.residual_out, a.qx, a.sx);      \
        return hipGetLastError();                                                                                 \
    }
    LQ_NORM(false, kNoRes) LQ_NORM(false, kResBf16) LQ_NORM(false, kResF32)
    LQ_NORM(true, kNoRes) LQ_NORM(true, kResBf16) LQ_NORM(true, kResF32)
#undef LQ_NORM
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rms_norm_int8(const NormArgs &args, hipStream_t st) {
    constexpr int64_t kSlice = int64_t(1) << 21;
    auto at = [](const void *p, int64_t bytes) { return p ? static_cast<const char *>(p) + bytes : nullptr; };
    for (int64_t row = 0; row < args.t; row += kSlice) {
        NormArgs a = args;
        const int64_t e = row * a.k;
        a.t = args.t - row < kSlice ? args.t - row : kSlice;
        a.x = at(args.x, e * (a.x_f32 ? 4 : 2));
        a.residual = at(args.residual, e * (a.residual_f32 ? 4 : 2));
        a.residual_out = const_cast<char *>(at(args.residual_out, e * (a.residual_f32 ? 4 : 2)));
        a.qx = args.qx + e;
        a.sx = args.sx + row;
        const hipError_t err = a.k <= 8192    ? launch_shape<256, 4, true>(a, st)
                               : a.k <= 32768 ? launch_shape<1024, 4, true>(a, st)
                                              : launch_shape<1024, 4, false>(a, st);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace lq
