// evict.hip -- eviction from the paged cache by accumulated attention weight
// (kv_cache_evict): each sequence and key head keeps its last tokens and the
// heaviest of the others.
//
// evict_select_kernel finds the positions that stay, a block a sequence and
// head: the weights' bits, mapped so that they order as the weights do, are
// narrowed down to the lightest one that stays in three passes over a histogram
// of 11 or 10 bits; two more passes count and write the positions in order.
// evict_move_kernel moves codes, scales, zeros and weights to the front of the
// table's pages. In place tokens move to earlier positions or stay, in order: a
// batch of tokens is read whole before any of it is written, and what later
// batches read lies behind what earlier ones write, so one block takes all tokens
// of a sequence and head, or of some bytes of their codes. Into other pages
// batches are shared out as well, unless some of them are the sequence's own. Bound
// by HBM with scattered rows of 64 or 128 bytes and quads of values of which one
// token in two to four stays: 16 sequences of up to 8192 tokens to 2048, 8 heads,
// INT8, 53 us for 178 MB, 3.4 TB/s; 6 of up to 30000 to 4000, 32 heads, INT4, 109 us
// for 437 MB, 4.0 TB/s (three sets of inputs in turn; one set again and again, which
// the last cache holds in part, 33 and 93, and in place 39 and 97).
#include "common.hpp"
#include "kv.hpp"

namespace lq {

namespace {

constexpr int kHeld = 32;  // weights a thread holds; longer sequences read the others anew
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

template <int THREADS>
__global__ __launch_bounds__(THREADS) void evict_select_kernel(EvictArgs a) {
    __shared__ uint32_t bins[kBins];
    __shared__ uint32_t sums[2][THREADS / 64];
    __shared__ uint32_t found[3];  // the digit, how many heavier weights stay, whether all of its do
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = blockIdx.x % a.c.heads;
    const int64_t seq = blockIdx.x / a.c.heads;
    const int len = (int)held_of(a, seq), keep = (int)a.keep, recent = (int)a.recent;
    int32_t *const kept = a.kept + ((int64_t)seq * a.c.heads + h) * a.keep;
    for (int i = (len < keep ? len : keep) + threadIdx.x; i < keep; i += THREADS) kept[i] = -1;
    if (len <= keep) {
        for (int i = threadIdx.x; i < len; i += THREADS) kept[i] = i;
        return;
    }
    const int old = len - recent;  // positions to choose among
    const uint32_t want = (uint32_t)(keep - recent);
    for (int i = threadIdx.x; i < recent; i += THREADS) kept[want + i] = old + i;
    if (want == 0) return;

    // A wave a run of positions, 64 side by side at a time.
    const int groups = (old + THREADS - 1) / THREADS, first = wave * groups * 64 + lane;
    const int32_t *const table = a.table + seq * a.max_pages;
    const int shift = a.c.page_shift, mask = (1 << shift) - 1;
    const int pages = (int)a.c.pages;
    auto weight = [&](int page, int i) {
        const bool in = (uint32_t)page < (uint32_t)pages;
        const float w = a.weights[(((int64_t)(in ? page : 0) * a.c.heads + h) << shift) + (i & mask)];
        return in ? order_of(w) : 0u;  // a position outside the pool goes first
    };
    // Places of the run behind the last position hold 0 as well: of equal ones
    // they come last, and there are enough before them.
    uint32_t u[kHeld] = {};
    int entry[kHeld / 16];  // pages of 1024 positions, at most 64, one a lane
#pragma unroll
    for (int c = 0; c < kHeld / 16; ++c) {
        const int page0 = ((first - lane) >> shift) + (1024 * c >> shift) + lane, last = (old - 1) >> shift;
        entry[c] = 16 * c < groups ? table[page0 < last ? page0 : last] : 0;
    }
    uint32_t none = 0;  // bit r: u[r] is no weight
#pragma unroll
    for (int r0 = 0; r0 < kHeld; r0 += 4)
        if (r0 < groups) {  // no load is waited for here
#pragma unroll
            for (int r = r0; r < r0 + 4; ++r) {
                const int i = first + 64 * r, page0 = ((first - lane) >> shift) + (1024 * (r / 16) >> shift);
                const int page = __shfl(entry[r / 16], (i >> shift) - page0);
                const bool in = (uint32_t)page < (uint32_t)pages;
                u[r] = __float_as_uint(a.weights[(((int64_t)(in ? page : 0) * a.c.heads + h) << shift) + (i & mask)]);
                none |= (in && i < old ? 0u : 1u) << r;
            }
        }
#pragma unroll
    for (int r0 = 0; r0 < kHeld; r0 += 4)
        if (r0 < groups) {
#pragma unroll
            for (int r = r0; r < r0 + 4; ++r) u[r] = (none >> r) & 1u ? 0u : order_of(__uint_as_float(u[r]));
        }
    // f(position's weight, position) for all of the wave's
    auto each = [&](auto f) {
#pragma unroll
        for (int r = 0; r < kHeld; ++r)
            if (r < groups) f(u[r], first + 64 * r);
        for (int r = kHeld; r < groups; ++r) {
            const int i = first + 64 * r, c = i < old ? i : old - 1;
            f(i < old ? weight(table[c >> shift], c) : 0u, i);
        }
    };

    uint32_t known = 0, known_mask = 0, need = want;
    for (int pass = 0; pass < 3; ++pass) {
        const int down = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit = pass < 2 ? kBins - 1 : kBins / 2 - 1;
        for (int i = threadIdx.x; i < kBins; i += THREADS) bins[i] = 0;
        __syncthreads();
        each([&](uint32_t x, int) {
            if ((x & known_mask) == known) atomicAdd(&bins[(x >> down) & digit], 1u);
        });
        __syncthreads();
        // runs of bins a thread, from the heaviest down: the one where the count
        // passes need
        constexpr int PER = kBins / THREADS;
        uint32_t n[PER], upto = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) upto += n[i] = bins[kBins - 1 - PER * threadIdx.x - i];
        const uint32_t mine = upto;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t v = __shfl_up(upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 63) sums[0][wave] = upto;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) upto += w < wave ? sums[0][w] : 0;
        uint32_t heavier = upto - mine;
        if (heavier < need && upto >= need) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (heavier < need && heavier + n[i] >= need) {
                    found[0] = kBins - 1 - PER * threadIdx.x - i;
                    found[1] = heavier;
                    found[2] = heavier + n[i] == need;
                }
                heavier += n[i];
            }
        }
        __syncthreads();
        known |= found[0] << down;
        known_mask |= digit << down;
        need -= found[1];
        if (found[2] && known != 0) {  // all with these digits stay: all above the next lower number
            known -= 1;
            need = 0;
            break;
        }
    }
    // All weights above `known` stay, and the first `need` of those equal to it:
    // counts of the waves' runs, then places.
    uint32_t above = 0, equal = 0;
    each([&](uint32_t x, int) {
        above += __popcll(__ballot(x > known));
        equal += __popcll(__ballot(x == known));
    });
    if (lane == 0) {
        sums[0][wave] = above;
        sums[1][wave] = equal;
    }
    __syncthreads();
    above = equal = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        above += w < wave ? sums[0][w] : 0;
        equal += w < wave ? sums[1][w] : 0;
    }
    each([&](uint32_t x, int i) {
        const uint64_t gt = __ballot(x > known), eq = __ballot(x == known);
        const uint32_t e = equal + lanes_below(eq);
        const uint32_t to = above + lanes_below(gt) + (e < need ? e : need);
        if (x > known || (x == known && e < need)) kept[to] = i;
        above += __popcll(gt);
        equal += __popcll(eq);
    });
}

// How the moving is shared out: blocks of a sequence and head take the 4-byte
// numbers, one of `keys` parts of the keys' code bytes or one of `values` parts
// of the values', of every `splits`th batch of tokens.
struct Shares {
    int keys, values, splits;
};
constexpr int kMove = 512;
constexpr int kBatch = 1024;  // tokens

template <int ROW>  // code bytes of a token
__global__ __launch_bounds__(kMove) void evict_move_kernel(EvictArgs a, Shares sh) {
    __shared__ int64_t from[kBatch], to[kBatch];  // slots of the head's tokens, or -1
    __shared__ int own;                           // to_table has pages of the table
    const int roles = 1 + sh.keys + sh.values;
    const int h = blockIdx.x % a.c.heads;
    const int role = blockIdx.x / a.c.heads % roles;
    const int split = blockIdx.x / a.c.heads / roles % sh.splits;
    const int64_t seq = blockIdx.x / a.c.heads / roles / sh.splits;
    const int64_t len = held_of(a, seq);
    const int count = (int)(len < a.keep ? len : a.keep);  // the same of new_lens
    if (role == 0 && h == 0 && split == 0 && threadIdx.x == 0) a.new_lens[seq] = count;
    const int32_t *const kept = a.kept + ((int64_t)seq * a.c.heads + h) * a.keep;
    // all stays where it is; by the positions, as new_lens may be the lengths
    if (a.to_table == a.table && (count == 0 || kept[count - 1] == count - 1)) return;
    const int32_t *const table = a.table + seq * a.max_pages, *const to_table = a.to_table + seq * a.to_pages;
    const int shift = a.c.page_shift, mask = (1 << shift) - 1;
    auto slot_of = [&](const int32_t *tab, int pos) -> int64_t {
        const int64_t page = tab[pos >> shift];
        return page < 0 || page >= a.c.pages ? -1 : ((page * a.c.heads + h) << shift) + (pos & mask);
    };
    // to_table may hold some of the table's pages, in their own places: what a batch
    // writes there lies before what later ones read, and one block takes them all.
    // Found out beside the first batch's lookups, for half a microsecond of 47
    // or 109 (one or two in front of them).
    bool ask = sh.splits > 1 && count > kBatch;
    int splits = sh.splits;
    if (threadIdx.x == 0) own = 0;
    for (int64_t at = (int64_t)split * kBatch; at < count; at += (int64_t)splits * kBatch) {
        const int j0 = (int)at, n = count - j0 < kBatch ? count - j0 : kBatch;
        __syncthreads();  // nobody reads the last lookups any more
#pragma unroll
        for (int u = 0; u < kBatch / kMove; ++u) {
            const int i = threadIdx.x + u * kMove;
            if (i < n) {
                from[i] = slot_of(table, kept[j0 + i]);
                to[i] = slot_of(to_table, j0 + i);
            }
        }
        if (ask)
            for (int i = threadIdx.x; i <= (count - 1) >> shift; i += kMove)
                if (table[i] == to_table[i]) own = 1;
        __syncthreads();
        if (ask && own) {
            if (split > 0) return;
            splits = 1;
        }
        ask = false;
        if (role == 0) {
            float *const src[5] = {a.weights, a.c.k_scales, a.c.v_scales, a.c.k_zeros, a.c.v_zeros};
            const int arrays = a.c.symmetric ? 3 : 5;
            float v[kBatch / kMove][5];
#pragma unroll
            for (int u = 0; u < kBatch / kMove; ++u) {
                const int i = threadIdx.x + u * kMove;
#pragma unroll
                for (int x = 0; x < 5; ++x)
                    if (x < arrays && i < n && from[i] >= 0) v[u][x] = src[x][from[i]];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kBatch / kMove; ++u) {
                const int i = threadIdx.x + u * kMove;
#pragma unroll
                for (int x = 0; x < 5; ++x)
                    if (x < arrays && i < n && from[i] >= 0 && to[i] >= 0) src[x][to[i]] = v[u][x];
            }
        } else if (role <= sh.keys) {
            constexpr int U = 4;
            const int width = ROW / 16 / sh.keys;                      // threads a token
            const int c = threadIdx.x % width + (role - 1) * width, t = threadIdx.x / width, step = kMove / width;
            for (int i0 = 0; i0 < n; i0 += U * step) {
                u32x4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + t + u * step;
                    if (i < n && from[i] >= 0) v[u] = *reinterpret_cast<const u32x4 *>(a.c.k_codes + from[i] * ROW + 16 * c);
                }
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + t + u * step;
                    if (i < n && from[i] >= 0 && to[i] >= 0)
                        *reinterpret_cast<u32x4 *>(a.c.k_codes + to[i] * ROW + 16 * c) = v[u];
                }
            }
        } else {
            // Four tokens of a quad and 16 bytes of their words a thread: byte o of
            // each word is token o's. Behind the last token the last one again.
            constexpr int U = 2;
            const int width = ROW / 4 / sh.values;
            const int c = threadIdx.x % width + (role - 1 - sh.keys) * width, t = threadIdx.x / width, step = kMove / width;
            for (int q0 = 0; 4 * q0 < n; q0 += U * step) {
                u32x4 w[U][4];
                int64_t s[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        const int i = 4 * (q0 + t + u * step) + o;
                        s[u][o] = from[i < n ? i : n - 1];
                        w[u][o] = *reinterpret_cast<const u32x4 *>(a.c.v_codes + (s[u][o] < 0 ? 0 : s[u][o] >> 2) * (4 * ROW) + 16 * c);
                    }
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = 4 * (q0 + t + u * step);
                    // selectors of two bytes each: the first token's, then the other's
                    const uint32_t s01 = 0x0C0C0400u + (uint32_t)(s[u][0] & 3) + ((uint32_t)(s[u][1] & 3) << 8);
                    const uint32_t s23 = 0x04000C0Cu + ((uint32_t)(s[u][2] & 3) << 16) + ((uint32_t)(s[u][3] & 3) << 24);
                    u32x4 v;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        v[x] = __builtin_amdgcn_perm(w[u][1][x], w[u][0][x], s01) | __builtin_amdgcn_perm(w[u][3][x], w[u][2][x], s23);
                    if (i < n && to[i] >= 0) *reinterpret_cast<u32x4 *>(a.c.v_codes + (to[i] >> 2) * (4 * ROW) + 16 * c) = v;
                }
            }
        }
    }
}

}  // namespace

template <int ROW>
static hipError_t launch_move(const EvictArgs &a, hipStream_t st) {
    const int64_t pairs = a.b * a.c.heads, room = a.max_pages << a.c.page_shift;
    int64_t kv = a.max_kv <= 0 || a.max_kv > room ? room : a.max_kv;
    if (kv > a.keep) kv = a.keep;  // tokens that may move
    Shares sh{1, 1, 1};
    // Two blocks of 512 threads a CU and a few rounds of them: values first, which
    // read four bytes for one. Of one set of inputs, what stayed read back after each
    // call: 1, 2 and 4 parts of each without batches side by side,
    // 16 sequences to 2048 tokens 56, 56 and 53 us, 47 with 2 and 2 and two batches
    // (this), 49 with 2 and 4; 6 to 4000 118, 121 and 129, 108 with 1 and 2 and four
    // batches (this), 119 with 2 and 4. 256 and 1024 threads 51 and 114, 51 and 115.
    while (sh.values < ROW / 16 && pairs * (sh.keys + sh.values) < 512) {
        if (sh.keys < sh.values && sh.keys < ROW / 32) sh.keys *= 2;
        else sh.values *= 2;
    }
    if (a.to_table != a.table) {
        const int64_t most = (kv + kBatch - 1) / kBatch;  // a batch a block
        const int64_t fill = 2048 / (pairs * (sh.keys + sh.values)) + 1;
        sh.splits = (int)(fill < most ? fill : most < 1 ? 1 : most);
    }
    const uint32_t blocks = (uint32_t)(pairs * (1 + sh.keys + sh.values) * sh.splits);
    hipLaunchKernelGGL(evict_move_kernel<ROW>, dim3(blocks), dim3(kMove), 0, st, a, sh);
    return hipGetLastError();
}

template <int THREADS>
static hipError_t launch_select(const EvictArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(evict_select_kernel<THREADS>, dim3((uint32_t)(a.b * a.c.heads)), dim3(THREADS), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_kv_evict(const EvictArgs &a, hipStream_t st) {
    // Fewer waves meet at fewer barriers, more hold longer sequences. 256, 512
    // and 1024 threads: 1003 tokens 6.4, 7.8 and 8.7 us; up to 8192 (16 sequences
    // of 8 heads) 17.7, 15.0 and 16.3; up to 30000 (6 of 32) 180, 74 and 28.
    const int64_t room = a.max_pages << a.c.page_shift, kv = a.max_kv <= 0 || a.max_kv > room ? room : a.max_kv;
    hipError_t e = kv <= 4096 ? launch_select<256>(a, st) : kv <= 512 * kHeld ? launch_select<512>(a, st)
                                                                              : launch_select<1024>(a, st);
    if (e != hipSuccess) return e;
    switch (a.c.head_dim * a.c.bits / 8) {
        case 32: return launch_move<32>(a, st);
        case 64: return launch_move<64>(a, st);
        case 128: return launch_move<128>(a, st);
        default: return launch_move<256>(a, st);
    }
}

}  // namespace lq
