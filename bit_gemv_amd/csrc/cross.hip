// cross.hip -- attention over the quantized paged cache beside paged_attention,
// by its kernels (attention.hpp): of rows that are no tokens of their sequence
// (cross_attention), and behind prefixes that sequences share (prefix_attention).
#include "attention.hpp"

namespace lq {

hipError_t launch_cross_attention(const AttnCall &a, hipStream_t st) { return launch_one<true>(a, plan_of(a), st); }

namespace {

// ---- attention over a shared prefix and over a sequence's own tokens ----
//
// The prefix's keys are read once for all rows that share it: its pass takes
// them as the rows of one sequence that each see everything, in tiles as a
// prompt's rows are. The own tokens' pass is paged_attention's. Both leave whole
// units as rows relative to their maximum and cut ones as parts, and
// attn_finish_kernel joins what either has of a row: one launch of 12 us for 64
// sequences of 64 heads, where joins of each pass and a merge took 26, and of 7 for
// 4, where they took 17. 64 rows behind 8192 shared tokens: own tokens (up to 1024
// each) 22 us, bound by HBM, the prefix 38, of 70 in all.
struct Launched {
    Span span;
    int log_tile, step;  // rows of a tile (log2), keys of a step
};
struct Source {
    KvBatch batch;
    Launched launch[2];
    int launches, whole;
    const float *o, *ml;  // whole units' rows
};

// Where a row's parts are: its sequence's units in their launch.
struct Found {
    int which;         // launch, or -1: the row belongs to no sequence
    int64_t begin, end;  // the sequence's rows
    uint32_t tiles;
    int steps;         // of a unit
    int64_t start, share;
};
// x0: the first 64 sequences' rows, a lane each
LQ_DEVICE Found find_row(const Source &s, const KvRows &x0, int64_t row, int shift, int group, int lane) {
    const KvBatch &bt = s.batch;
    Found f{-1, 0, 0, 0, 0, 0, 0};
    int64_t seq = -1;
    uint32_t rows = 0;
    for (int64_t s0 = 0; s0 < bt.b && seq < 0; s0 += 64) {
        KvRows x = x0;
        if (s0 > 0) x = s0 + lane < bt.b ? kv_rows(bt, s0 + lane, shift, s.whole) : KvRows{0, 0, 0, 0};
        const uint64_t in = __ballot(row >= x.begin && row < x.begin + x.n);
        if (in) {
            const int src = __ffsll((unsigned long long)in) - 1;
            seq = s0 + src;
            f.begin = readlane64(x.begin, src);
            f.end = f.begin + readlane64(x.n, src);
            rows = (uint32_t)(f.end - f.begin) * (uint32_t)group;
        }
    }
    if (seq < 0) return f;
    f.which = s.launches == 2 && rows <= s.launch[1].span.most ? 1 : 0;
    const Launched &l = s.launch[f.which];
    f.tiles = (rows + (1u << l.log_tile) - 1) >> l.log_tile;
    int64_t sum = 0;  // as Schedule adds the sequences' steps up
    for (int64_t s0 = 0; s0 < bt.b; s0 += 64) {
        KvRows x = x0;
        if (s0 > 0) x = s0 + lane < bt.b ? kv_rows(bt, s0 + lane, shift, s.whole) : KvRows{0, 0, 0, 0};
        int64_t all = 0;
        int steps = 1;
        const uint32_t n = (uint32_t)x.n * (uint32_t)group;
        if (s0 + lane < bt.b && n >= l.span.least && n <= l.span.most) {
            int64_t keys = x.first + x.n < x.len ? x.first + x.n : x.len;
            keys = keys < 1 ? 1 : keys;
            steps = l.span.form & kByUnit ? 1 : (int)((keys + l.step - 1) / l.step);
            all = (int64_t)((n + (1u << l.log_tile) - 1) >> l.log_tile) * steps;
        }
        const int64_t upto = sum + scan64(all);
        if (seq >= s0 && seq < s0 + 64) {
            f.steps = __builtin_amdgcn_readlane(steps, (int)(seq - s0));
            f.start = readlane64(upto - all, (int)(seq - s0));
        }
        sum = readlane64(upto, 63);
    }
    f.share = uniform_div(sum + l.span.cap - 1, l.span.cap);
    return f;
}

LQ_DEVICE int64_t lane_div(int64_t a, int64_t b) {  // a >= 0, b > 0, other numbers in other lanes
    return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The parts of a row and head in one source: how many, and the i-th's row of
// floats and its maximum and sum.
struct Parts {
    const float *o, *ml;  // the first one
    int64_t next;         // to the second one, in rows
    int64_t step;         // from each to the next
    int n;
};
template <int D>
LQ_DEVICE Parts parts_of(const Source &s, const Found &f, int64_t row, const AttnArgs &a, int group, int h, int head) {
    if (f.which < 0) return Parts{nullptr, nullptr, 0, 0, 0};
    const Launched &la = s.launch[f.which];
    const uint32_t rr = (uint32_t)(row - f.begin) * (uint32_t)group + head;
    const uint32_t tile = rr >> la.log_tile, r = rr & ((1u << la.log_tile) - 1);
    // the unit's place among its sequence's, as Schedule orders them
    const uint32_t j = la.span.form & kByUnit ? f.tiles - 1 - tile : 2 * tile < f.tiles ? 2 * tile : 2 * (f.tiles - 1 - tile) + 1;
    const int64_t start = f.start + (int64_t)j * f.steps;
    const int64_t first = lane_div(start, f.share), last = lane_div(start + f.steps - 1, f.share);
    const bool whole = first == last;
    // the unit's first part is its block's first piece if it starts there
    const int64_t second_place = start > first * f.share;
    const int64_t at = whole ? row * a.q_heads + h * group + head
                             : (((2 * first + second_place) * a.c.heads + h) << la.log_tile) + r;
    const int64_t place = (int64_t)a.c.heads << la.log_tile;  // rows of a block's piece
    return Parts{(whole ? s.o : la.span.o) + at * D, (whole ? s.ml : la.span.ml) + at * 2, (2 - second_place) * place,
                 2 * place, (int)(last - first) + 1};
}

// m, l and v (lane c's four elements) of a row and head over its parts in both
// sources, or over those of one of `takers`.
LQ_DEVICE void join_row(const Parts &x, const Parts &y, int d, int c, int taker, int takers, float &m, float &l, f32x4 &v) {
    constexpr int U = 8;  // parts in flight
    m = -1e30f;
    l = 0.0f;
    v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int parts = x.n + y.n;
    for (int i0 = taker; i0 < parts; i0 += U * takers) {
        float2 ml[U];
        f32x4 p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * takers;
            const bool of_x = i < x.n;
            const int k = of_x ? i : i - x.n;
            const int64_t rows = k == 0 ? 0 : (of_x ? x.next : y.next) + (int64_t)(k - 1) * (of_x ? x.step : y.step);
            ml[u] = float2{-__builtin_inff(), 0.0f};
            p[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (i < parts) {
                ml[u] = *reinterpret_cast<const float2 *>((of_x ? x.ml : y.ml) + rows * 2);
                p[u] = *reinterpret_cast<const f32x4 *>((of_x ? x.o : y.o) + rows * d + 4 * c);
            }
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u].x);
        const float by = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= by;
        v *= by;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = __builtin_amdgcn_exp2f(ml[u].x - mn);
            l = __builtin_fmaf(ml[u].y, w, l);
            v += p[u] * w;
        }
    }
}

// D / 4 lanes a row and head. Blocks take `run` rows of a key head and its group;
// SPLIT: a block a row and head, whose parts its teams share.
template <int D, bool SPLIT>
__global__ __launch_bounds__(256) void attn_finish_kernel(AttnArgs a, Source own, Source prefix, int run) {
    constexpr int W = D / 4, TEAMS = 256 / W;
    __shared__ f32x4 lds_v[SPLIT ? TEAMS : 1][W];
    __shared__ float2 lds_ml[TEAMS];
    const int lane = threadIdx.x & 63, team = threadIdx.x / W, c = threadIdx.x % W;
    const int heads = SPLIT ? a.q_heads : a.c.heads, group = a.q_heads / a.c.heads, shift = a.c.page_shift;
    const KvRows none{0, 0, 0, 0};
    const KvRows x0 = lane < own.batch.b ? kv_rows(own.batch, lane, shift) : none;
    const KvRows y0 = lane < prefix.batch.b ? kv_rows(prefix.batch, lane, shift, prefix.whole) : none;
    const int h = SPLIT ? blockIdx.x % heads / group : blockIdx.x % heads;
    int64_t row = (int64_t)(blockIdx.x / heads) * run;
    const int64_t end = row + run < a.batch.rows ? row + run : a.batch.rows;
    while (row < end) {
        // rows up to the end of a sequence, of the own rows or of the prefix's
        const Found mine = find_row(own, x0, row, shift, group, lane);
        const Found shared = find_row(prefix, y0, row, shift, group, lane);
        int64_t until = mine.which < 0 || shared.which < 0 ? row + 1 : mine.end < shared.end ? mine.end : shared.end;
        until = until < end ? until : end;
        const int items = mine.which < 0 ? 0 : SPLIT ? TEAMS : (int)(until - row) * group;
        for (int i = team; i < items; i += TEAMS) {
            const int64_t my_row = SPLIT ? row : row + i / group;
            const int head = SPLIT ? blockIdx.x % heads % group : i % group;
            const int64_t at = my_row * a.q_heads + h * group + head;
            float m, l;
            f32x4 v;
            join_row(parts_of<D>(own, mine, my_row, a, group, h, head), parts_of<D>(prefix, shared, my_row, a, group, h, head),
                     D, c, SPLIT ? team : 0, SPLIT ? TEAMS : 1, m, l, v);
            if constexpr (SPLIT) {
                lds_v[team][c] = v;
                if (c == 0) lds_ml[team] = float2{m, l};
                __syncthreads();
                if (team > 0) continue;
#pragma unroll
                for (int t = 1; t < TEAMS; ++t) m = fmaxf(m, lds_ml[t].x);
                l = 0.0f;
                v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int t = 0; t < TEAMS; ++t) {
                    const float w = __builtin_amdgcn_exp2f(lds_ml[t].x - m);
                    l = __builtin_fmaf(lds_ml[t].y, w, l);
                    v += lds_v[t][c] * w;
                }
            }
            v *= inverse_sum(l);
            const bf16x2_t b0{(__bf16)v[0], (__bf16)v[1]}, b1{(__bf16)v[2], (__bf16)v[3]};
            *reinterpret_cast<u32x2 *>(a.out + at * D + 4 * c) =
                u32x2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
            if (c == 0 && a.lse) a.lse[at] = log_sum(m, l);
        }
        row = until;
    }
}

}  // namespace

static int64_t part_bytes(int64_t rows, int64_t q_heads, int64_t floats) {
    return (rows * q_heads * floats * 4 + 255) / 256 * 256;
}

int64_t prefix_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t page_size,
                               int64_t p, int64_t prefix_pages, int64_t max_prefix_rows, int64_t max_prefix, int64_t b,
                               int64_t max_pages, int64_t max_rows, int64_t max_kv) {
    const int64_t own = attention_workspace_bytes(rows, q_heads, heads, head_dim, b, max_pages, page_size, max_rows,
                                                  max_kv, false);
    if (p == 0) return own;
    return own + 2 * (part_bytes(rows, q_heads, head_dim) + part_bytes(rows, q_heads, 2)) +
           attention_workspace_bytes(rows, q_heads, heads, head_dim, p, prefix_pages, page_size, max_prefix_rows,
                                     max_prefix, true);
}

hipError_t launch_prefix_attention(const PrefixArgs &a, hipStream_t st) {
    if (a.prefix.b == 0) return launch_paged_attention(a.own, st);
    AttnCall side[2] = {a.own, a.own};
    side[1].batch = a.prefix;
    side[1].whole = 1;
    side[1].max_rows = a.max_prefix_rows;
    side[1].max_kv = a.max_prefix;
    Source source[2];
    char *ws = static_cast<char *>(a.own.workspace);
    for (int i = 0; i < 2; ++i) {
        AttnCall &x = side[i];
        x.apart = 1;
        x.out = reinterpret_cast<uint16_t *>(ws);
        x.lse = reinterpret_cast<float *>(ws + part_bytes(x.batch.rows, x.q_heads, x.c.head_dim));
        const Plan p = plan_of(x);
        ws += part_bytes(x.batch.rows, x.q_heads, x.c.head_dim) + part_bytes(x.batch.rows, x.q_heads, 2);
        x.workspace = ws;
        ws += p.bytes;
        Source &s = source[i];
        s.batch = x.batch;
        s.launches = p.passes;
        s.whole = x.whole;
        s.o = reinterpret_cast<float *>(x.out);
        s.ml = x.lse;
        for (int k = 0; k < p.passes; ++k) {
            const Pass &q = p.pass[k];
            s.launch[k] = {span_of(x, q, static_cast<char *>(x.workspace) + (k ? p.pass[0].bytes : 0)),
                           __builtin_ctz(q.row_tile),
                           q.row_tile < 128 ? kFewStep : q.row_tile / (x.c.head_dim == 64 ? 2 : 4)};
        }
        const hipError_t e = launch_one<true>(x, p, st);
        if (e != hipSuccess) return e;
    }
    // Few rows: teams beside each other for the parts as well. With and without,
    // rows of 64 / 8 heads: 4 behind 2011 tokens 24.5 and 32.3 us a call, 16 behind
    // 4096 48.0 and 50.7, 64 behind 8192 94.0 and 74.8. 2048, 1024 and 512 blocks of
    // 439296 threads' work: 19.3, 21.7 and 26.2.
    const int64_t rows = a.own.batch.rows, heads = a.own.c.heads;
    auto finish = [&](auto split_kernel, auto kernel) {
        if (rows * a.own.q_heads <= 1024) {
            hipLaunchKernelGGL(split_kernel, dim3((uint32_t)(rows * a.own.q_heads)), dim3(256), 0, st, a.own, source[0],
                               source[1], 1);
        } else {
            const int64_t blocks = 2048 / heads + 1, run = (rows + blocks - 1) / blocks;
            hipLaunchKernelGGL(kernel, dim3((uint32_t)((rows + run - 1) / run * heads)), dim3(256), 0, st, a.own, source[0],
                               source[1], (int)run);
        }
        return hipGetLastError();
    };
    return a.own.c.head_dim == 64    ? finish(attn_finish_kernel<64, true>, attn_finish_kernel<64, false>)
           : a.own.c.head_dim == 128 ? finish(attn_finish_kernel<128, true>, attn_finish_kernel<128, false>)
                                     : finish(attn_finish_kernel<256, true>, attn_finish_kernel<256, false>);
}

}  // namespace lq
