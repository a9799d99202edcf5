// w4a16_paged_attention: the workspace and the choice by the cache's type.
#include "paged_attention.h"

namespace w4a16 {

bool attention_costs_fit(int most, int window, int q_heads, int kv_heads) {
    // (256 dims may take two rows of 8 for 16 heads, but over a short cache only)
    const int heads = q_heads / kv_heads > 8 ? 16 : 8;
    return (static_cast<int64_t>(most_tiles(most, window)) + kRowCost) * rows_of_request(q_heads, kv_heads, heads) <= kMostCost;
}

size_t paged_attention_workspace(int q_heads, int kv_heads, int dim) {
    const int heads = q_heads / kv_heads > 8 ? 16 : 8, padded = padded_dim(dim);
    return static_cast<size_t>(most_workers(padded)) *
           (sizeof(int4) + 2 * static_cast<size_t>(heads) * (padded + 2) * sizeof(float));
}

cudaError_t launch_paged_attention(const AttentionArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    JoinPlan join{};
    join.joins = static_cast<int4*>(a.workspace);
    join.part = reinterpret_cast<float*>(join.joins + most_workers(padded_dim(a.cache.dim)));
    return a.cache.dtype == W4A16_CACHE_BF16 ? launch_attention_bf16(a, dev, join, s)
                                             : launch_attention_e4m3(a, dev, join, s);
}

}  // namespace w4a16
