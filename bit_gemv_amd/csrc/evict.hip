// evict.hip -- eviction from the paged cache by accumulated attention weight
// (kv_cache_evict): each sequence and key head keeps its last tokens and the
// heaviest of the others.
//
// evict_select_kernel finds the positions that stay, a block a sequence and
// head: the weights' bits, mapped so that they order as the weights do, are
// narrowed down to the lightest one that stays in three passes over a histogram
// of 11 or 10 bits; two more passes count and write the positions in order.
// evict_move_kernel moves codes, scales, zeros and weights to the front of the
// table's pages. Its tokens move to earlier positions or stay, in order: a batch
// of tokens is read whole before any of it is written, and what later batches
// read lies behind what earlier ones write, so a table may be its own target.
#include "common.hpp"
#include "kv.hpp"

namespace lq {

namespace {

constexpr int kSelect = 1024;   // threads of a selecting block
constexpr int kHeld = 32768;    // weights held in LDS; longer sequences read the others anew
constexpr int kBins = 2048;

// Weights as unsigned numbers that order as they do, -0 as 0; NaN is heaviest.
LQ_DEVICE uint32_t order_of(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

LQ_DEVICE int64_t held_of(const EvictArgs &a, int64_t seq) {
    const int64_t room = a.max_pages << a.c.page_shift, held = a.lens[seq];
    return held < 0 ? 0 : held < room ? held : room;
}

LQ_DEVICE int lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

__global__ __launch_bounds__(kSelect) void evict_select_kernel(EvictArgs a) {
    __shared__ uint32_t held[kHeld];
    __shared__ uint32_t bins[kBins];
    __shared__ uint32_t sums[2][kSelect / 64];
    __shared__ uint32_t found[2];  // the digit, and how many heavier weights stay
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int h = blockIdx.x % a.c.heads;
    const int64_t seq = blockIdx.x / a.c.heads;
    const int64_t len = held_of(a, seq);
    int32_t *const kept = a.kept + ((int64_t)seq * a.c.heads + h) * a.keep;
    const int64_t left = len < a.keep ? len : a.keep;
    for (int64_t i = left + threadIdx.x; i < a.keep; i += kSelect) kept[i] = -1;
    if (len <= a.keep) {
        for (int64_t i = threadIdx.x; i < len; i += kSelect) kept[i] = (int32_t)i;
        return;
    }
    const int64_t old = len - a.recent;              // positions to choose among
    const uint32_t want = (uint32_t)(a.keep - a.recent);
    for (int64_t i = threadIdx.x; i < a.recent; i += kSelect) kept[want + i] = (int32_t)(old + i);
    if (want == 0) return;

    const int32_t *const table = a.table + seq * a.max_pages;
    const int shift = a.c.page_shift, mask = (1 << shift) - 1;
    auto weight = [&](int64_t i) {
        const int64_t page = table[i >> shift];
        // a position outside the pool goes first
        if (page < 0 || page >= a.c.pages) return 0u;
        return order_of(a.weights[((page * a.c.heads + h) << shift) + (i & mask)]);
    };
    const int64_t in_lds = old < kHeld ? old : kHeld;
    for (int64_t i = threadIdx.x; i < in_lds; i += kSelect) held[i] = weight(i);
    auto at = [&](int64_t i) { return i < kHeld ? held[i] : weight(i); };

    uint32_t known = 0, known_mask = 0, need = want;
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, down = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        for (int i = threadIdx.x; i < kBins; i += kSelect) bins[i] = 0;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < old; i += kSelect) {
            const uint32_t u = at(i);
            if ((u & known_mask) == known) atomicAdd(&bins[(u >> down) & (kBins - 1) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        // two bins a thread, from the heaviest down: the one where the count passes need
        const uint32_t hi = bins[kBins - 1 - 2 * threadIdx.x], lo = bins[kBins - 2 - 2 * threadIdx.x];
        uint32_t upto = hi + lo;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t v = __shfl_up(upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 63) sums[0][wave] = upto;
        __syncthreads();
        uint32_t before = 0;
        for (int w = 0; w < wave; ++w) before += sums[0][w];
        upto += before;
        const uint32_t heavier = upto - hi - lo;
        if (heavier < need && upto >= need) {
            const bool first = heavier + hi >= need;
            found[0] = kBins - (first ? 1 : 2) - 2 * threadIdx.x;
            found[1] = first ? heavier : heavier + hi;
        }
        __syncthreads();
        known |= found[0] << down;
        known_mask |= ((1u << bits) - 1) << down;
        need -= found[1];
    }
    // All weights above `known` stay, and the first `need` of those equal to it.
    // A wave a run of positions: counts, then places.
    const int64_t run = ((old + kSelect - 1) / kSelect) * 64, i0 = wave * run, i1 = i0 + run < old ? i0 + run : old;
    uint32_t above = 0, equal = 0;
    for (int64_t i = i0; i < i1; i += 64) {
        const uint32_t u = i + lane < i1 ? at(i + lane) : 0;
        above += __popcll(__ballot(i + lane < i1 && u > known));
        equal += __popcll(__ballot(i + lane < i1 && u == known));
    }
    if (lane == 0) {
        sums[0][wave] = above;
        sums[1][wave] = equal;
    }
    __syncthreads();
    above = equal = 0;
    for (int w = 0; w < wave; ++w) {
        above += sums[0][w];
        equal += sums[1][w];
    }
    for (int64_t i = i0; i < i1; i += 64) {
        const bool in = i + lane < i1;
        const uint32_t u = in ? at(i + lane) : 0;
        const uint64_t gt = __ballot(in && u > known), eq = __ballot(in && u == known);
        const uint32_t e = equal + lanes_below(eq);
        const uint32_t to = above + lanes_below(gt) + (e < need ? e : need);
        if (in && (u > known || (u == known && e < need))) kept[to] = (int32_t)(i + lane);
        above += __popcll(gt);
        equal += __popcll(eq);
    }
}

// What a block of evict_move_kernel moves: keys' codes, values' codes, or the
// 4-byte numbers.
enum { kKeys, kValues, kNumbers, kRoles };
constexpr int kMove = 256;

template <int ROW>  // code bytes of a token
__global__ __launch_bounds__(kMove) void evict_move_kernel(EvictArgs a) {
    const int h = blockIdx.x % a.c.heads;
    const int role = blockIdx.x / a.c.heads % kRoles;
    const int64_t seq = blockIdx.x / a.c.heads / kRoles;
    const int64_t len = held_of(a, seq);
    const int count = (int)(len < a.keep ? len : a.keep);
    if (role == kNumbers && h == 0 && threadIdx.x == 0) a.new_lens[seq] = count;
    if (len <= a.keep && a.to_table == a.table) return;  // all stays where it is
    const int32_t *const kept = a.kept + ((int64_t)seq * a.c.heads + h) * a.keep;
    const int32_t *const table = a.table + seq * a.max_pages, *const to_table = a.to_table + seq * a.to_pages;
    const int shift = a.c.page_shift, mask = (1 << shift) - 1;
    // slots of a head's token, or -1
    auto slot_of = [&](const int32_t *tab, int64_t pos) -> int64_t {
        const int64_t page = tab[pos >> shift];
        return page < 0 || page >= a.c.pages ? -1 : ((page * a.c.heads + h) << shift) + (pos & mask);
    };
    if (role == kKeys) {
        constexpr int TPT = ROW / 16, U = 4, T = kMove / TPT * U;  // threads a token, tokens a thread, tokens a batch
        const int c = threadIdx.x % TPT, t = threadIdx.x / TPT;
        for (int j0 = 0; j0 < count; j0 += T) {
            u32x4 v[U];
            int64_t to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + t + u * (kMove / TPT);
                to[u] = -1;
                if (j < count) {
                    const int64_t from = slot_of(table, kept[j]);
                    to[u] = slot_of(to_table, j);
                    if (from < 0) to[u] = -1;
                    else v[u] = *reinterpret_cast<const u32x4 *>(a.c.k_codes + from * ROW + 16 * c);
                }
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u] >= 0) *reinterpret_cast<u32x4 *>(a.c.k_codes + to[u] * ROW + 16 * c) = v[u];
        }
    } else if (role == kValues) {
        constexpr int TPQ = ROW / 4, U = 2, Q = kMove / TPQ * U;  // threads a quad of tokens (16 bytes each), ...
        const int c = threadIdx.x % TPQ, t = threadIdx.x / TPQ;
        for (int q0 = 0; 4 * q0 < count; q0 += Q) {
            u32x4 v[U];
            int64_t to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + t + u * (kMove / TPQ);
                to[u] = -1;
                v[u] = u32x4{0u, 0u, 0u, 0u};
                if (4 * q < count) {
                    to[u] = slot_of(to_table, 4 * q);
                    // byte o of each word is token 4 q + o's
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        const int j = 4 * q + o < count ? 4 * q + o : count - 1;
                        const int64_t from = slot_of(table, kept[j]);
                        if (from < 0) continue;
                        const u32x4 w = *reinterpret_cast<const u32x4 *>(a.c.v_codes + (from >> 2) * (4 * ROW) + 16 * c);
                        const int down = 8 * (int)(from & 3);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[u][i] |= ((w[i] >> down) & 255u) << (8 * o);
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u] >= 0) *reinterpret_cast<u32x4 *>(a.c.v_codes + (to[u] >> 2) * (4 * ROW) + 16 * c) = v[u];
        }
    } else {
        float *const src[5] = {a.weights, a.c.k_scales, a.c.v_scales, a.c.k_zeros, a.c.v_zeros};
        const int n = a.c.symmetric ? 3 : 5;
        for (int j0 = 0; j0 < count; j0 += kMove) {
            float v[5];
            int64_t from = -1, to = -1;
            const int j = j0 + threadIdx.x;
            if (j < count) {
                from = slot_of(table, kept[j]);
                to = slot_of(to_table, j);
            }
#pragma unroll
            for (int i = 0; i < 5; ++i)
                if (i < n && from >= 0) v[i] = src[i][from];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 5; ++i)
                if (i < n && from >= 0 && to >= 0) src[i][to] = v[i];
        }
    }
}

}  // namespace

hipError_t launch_kv_evict(const EvictArgs &a, hipStream_t st) {
    const uint32_t blocks = (uint32_t)(a.b * a.c.heads);
    hipLaunchKernelGGL(evict_select_kernel, dim3(blocks), dim3(kSelect), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    switch (a.c.head_dim * a.c.bits / 8) {
        case 32: hipLaunchKernelGGL(evict_move_kernel<32>, dim3(blocks * kRoles), dim3(kMove), 0, st, a); break;
        case 64: hipLaunchKernelGGL(evict_move_kernel<64>, dim3(blocks * kRoles), dim3(kMove), 0, st, a); break;
        case 128: hipLaunchKernelGGL(evict_move_kernel<128>, dim3(blocks * kRoles), dim3(kMove), 0, st, a); break;
        default: hipLaunchKernelGGL(evict_move_kernel<256>, dim3(blocks * kRoles), dim3(kMove), 0, st, a); break;
    }
    return hipGetLastError();
}

}  // namespace lq
