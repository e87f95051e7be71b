// kv.hpp -- the quantized paged KV cache as the kernels see it: arguments,
// addresses and the batch's rows. Layout: include/libquant.h, lq_kv_cache.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lq {

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // a table's room for one sequence: the kernels' keys are 32-bit

struct KvCache {
    uint8_t *k_codes, *v_codes;
    float *k_scales, *k_zeros, *v_scales, *v_zeros;
    int64_t pages;
    int page_shift;  // log2(page_size)
    int heads, head_dim, bits, symmetric;
};

struct KvBatch {
    const int32_t *table, *lens, *starts;
    int64_t b, max_pages, rows;
};

struct KvWriteArgs {
    KvCache c;
    KvBatch batch;
    const void *k, *v;
    int f32;
    int64_t k_stride, v_stride, max_rows;
    int flat = 0;  // set by the launcher: see kv_grid
};

struct KvReadArgs {
    KvCache c;
    KvBatch batch;
    void *k, *v;
    int f32;
    int64_t max_rows;
    int flat = 0;
};

struct AttnArgs {
    KvCache c;
    KvBatch batch;
    const uint16_t *q;
    int64_t q_stride;
    int q_heads;
    float scale;
    int64_t max_rows, max_kv;
    void *workspace;
    uint16_t *out;
    float *lse;
};

// A call, with the forms beside paged_attention's, which the kernels have in Span.
struct AttnCall : AttnArgs {
    int whole = 0;  // the rows are no tokens of the sequence: each sees all that it holds
    // For a result that is joined with another: whole units' rows relative to their
    // maximum, fp32, go to out, their maximum (log2) and sum to lse, [rows][q_heads][2];
    // cut units' parts stay in the workspace.
    int apart = 0;
};

// Attention over a prefix that several sequences share and over their own
// tokens: `own` is the whole call, `prefix` the groups of rows that share one.
struct PrefixArgs {
    AttnCall own;
    KvBatch prefix;
    int64_t max_prefix_rows, max_prefix;
};

// The attention weight that cached tokens receive; weights and out fp32 in the
// scales' layout, weights null: from zero.
struct WeighArgs {
    KvCache c;
    KvBatch batch;
    const uint16_t *q;
    int64_t q_stride;
    int q_heads;
    float scale;
    const float *lse, *weights;
    float *out;
    int64_t max_rows, max_kv;
    void *workspace;
    int whole;  // as AttnCall's
};

// Eviction by weight from the sequences' pages to the front of to_table's.
struct EvictArgs {
    KvCache c;
    float *weights;
    const int32_t *table, *lens;
    int64_t b, max_pages;
    int64_t keep, recent;
    const int32_t *to_table;
    int64_t to_pages;
    int64_t max_kv;
    int32_t *kept, *new_lens;
};

hipError_t launch_kv_write(const KvWriteArgs &a, hipStream_t st);
hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t st);
int64_t weigh_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t b, int64_t max_pages,
                              int64_t page_size, int64_t max_rows, int64_t max_kv);
hipError_t launch_kv_weigh(const WeighArgs &a, hipStream_t st);
hipError_t launch_kv_evict(const EvictArgs &a, hipStream_t st);
int64_t attention_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t b,
                                  int64_t max_pages, int64_t page_size, int64_t max_rows, int64_t max_kv, bool whole);
int64_t prefix_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t page_size,
                               int64_t p, int64_t prefix_pages, int64_t max_prefix_rows, int64_t max_prefix, int64_t b,
                               int64_t max_pages, int64_t max_rows, int64_t max_kv);
hipError_t launch_paged_attention(const AttnCall &a, hipStream_t st);  // neither whole nor apart
hipError_t launch_cross_attention(const AttnCall &a, hipStream_t st);
hipError_t launch_prefix_attention(const PrefixArgs &a, hipStream_t st);

// One sequence's rows: [begin, begin + n) of the row tensors, row begin + i at
// position first + i. Out-of-range starts are cut to the row tensors. Rows that
// see everything stand behind the last token.
struct KvRows {
    int64_t begin, n, first, len;  // len: tokens held, cut to the table
};

__device__ __forceinline__ KvRows kv_rows(const KvBatch &bt, int64_t seq, int page_shift, bool whole = false) {
    const int64_t s0 = bt.starts[seq], s1 = bt.starts[seq + 1], held = bt.lens[seq];
    KvRows r;
    r.begin = s0 < 0 ? 0 : s0;
    const int64_t end = s1 > bt.rows ? bt.rows : s1;
    r.n = end > r.begin ? end - r.begin : 0;
    const int64_t room = bt.max_pages << page_shift;
    r.len = held > room ? room : held;
    r.first = whole ? r.len : held - (s1 - r.begin);
    return r;
}

// The page of a sequence's token, or -1 where the table gives none in the pool.
__device__ __forceinline__ int64_t kv_page(const KvBatch &bt, int64_t seq, int64_t pos, int page_shift, int64_t pages) {
    const int64_t i = pos >> page_shift;
    if (pos < 0 || i >= bt.max_pages) return -1;
    const int64_t p = bt.table[seq * bt.max_pages + i];
    return p < 0 || p >= pages ? -1 : p;
}

// One lane's value, and quotients, as wave-uniform numbers.
__device__ __forceinline__ int64_t readlane64(int64_t v, int src) {
    const int lo = __builtin_amdgcn_readlane((int)v, src), hi = __builtin_amdgcn_readlane((int)(v >> 32), src);
    return ((int64_t)hi << 32) | (uint32_t)lo;
}
__device__ __forceinline__ int64_t uniform_div(int64_t a, int64_t b) {  // a >= 0, b > 0
    if ((a | b) >> 32) return a / b;
    return (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a / (uint32_t)b);
}

template <int CTRL, int ROWMASK>
__device__ __forceinline__ int64_t dpp_add64(int64_t v) {  // v plus the lane's source, or plus 0 where it has none
    const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWMASK, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWMASK, 0xF, false);
    return v + (((int64_t)hi << 32) | (uint32_t)lo);
}
// Inclusive sum over the wave's lanes: shifts by 1, 2, 4, 8 within rows of 16,
// then each row's last lane to the next row and lane 31 to the upper half.
__device__ __forceinline__ int64_t scan64(int64_t v) {
    v = dpp_add64<0x111, 0xF>(v);
    v = dpp_add64<0x112, 0xF>(v);
    v = dpp_add64<0x114, 0xF>(v);
    v = dpp_add64<0x118, 0xF>(v);
    v = dpp_add64<0x142, 0xA>(v);
    return dpp_add64<0x143, 0xC>(v);
}

}  // namespace lq
