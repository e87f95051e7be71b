// attention.hip -- causal attention of new tokens over the quantized paged
// cache (paged_attention): attention.hpp's kernels without the forms beside it.
#include "attention.hpp"

namespace lq {

int64_t attention_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t b,
                                  int64_t max_pages, int64_t page_size, int64_t max_rows, int64_t max_kv, bool whole) {
    // of either format: INT4's blocks are as many as INT8's or more
    return plan_of(rows, q_heads, heads, head_dim, 4, b, max_pages * page_size, max_rows, max_kv, whole).bytes;
}

hipError_t launch_paged_attention(const AttnCall &a, hipStream_t st) { return launch_one<false>(a, plan_of(a), st); }

}  // namespace lq
