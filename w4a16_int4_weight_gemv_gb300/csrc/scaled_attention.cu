// w4a16_scaled_attention: the workspace and the choice by the cache's type.
#include <algorithm>

#include "paged_attention.h"
#include "scaled.h"

namespace w4a16 {

// scaled_attention_e4m3.cu, scaled_attention_int8.cu and their *_wide.cu: all launches of a call
cudaError_t launch_attention_e4m3_groups(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);
cudaError_t launch_attention_int8_groups(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);
cudaError_t launch_attention_e4m3_groups_wide(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);
cudaError_t launch_attention_int8_groups_wide(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);

size_t scaled_attention_workspace(int q_heads, int kv_heads, int dim, int new_tokens) {
    // (fewer new tokens may be worked on in larger rows: 36 columns as 24 twice, 32 as they are)
    const int padded = padded_dim(dim), columns = std::min((q_heads / kv_heads * new_tokens + 7) / 8 * 8, most_together(dim));
    return static_cast<size_t>(most_workers(padded)) * (sizeof(int4) + 2 * static_cast<size_t>(columns) * (padded + 2) * sizeof(float));
}

cudaError_t launch_scaled_attention(const ScaledAttentionArgs& a, int int8, const DeviceInfo& dev, cudaStream_t s) {
    JoinPlan join{};
    join.joins = static_cast<int4*>(a.workspace);
    join.part = reinterpret_cast<float*>(join.joins + most_workers(padded_dim(a.cache.dim)));
    const bool wide = columns_together(a.q_heads / a.cache.heads * a.tokens, a.cache.dim) > 16;
    if (int8) return wide ? launch_attention_int8_groups_wide(a, dev, join, s) : launch_attention_int8_groups(a, dev, join, s);
    return wide ? launch_attention_e4m3_groups_wide(a, dev, join, s) : launch_attention_e4m3_groups(a, dev, join, s);
}

}  // namespace w4a16
