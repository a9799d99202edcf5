// w4a16_scaled_attention: the choice by the cache's type.
#include "paged_attention.h"
#include "scaled.h"

namespace w4a16 {

// scaled_attention_e4m3.cu, scaled_attention_int8.cu: all launches of a call
cudaError_t launch_attention_e4m3_groups(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);
cudaError_t launch_attention_int8_groups(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);

cudaError_t launch_scaled_attention(const ScaledAttentionArgs& a, int int8, const DeviceInfo& dev, cudaStream_t s) {
    JoinPlan join{};
    join.joins = static_cast<int4*>(a.workspace);
    const int padded = padded_dim(a.cache.dim), heads = a.q_heads / a.cache.heads * a.tokens > 8 ? 16 : 8;
    join.part = reinterpret_cast<float*>(join.joins + most_workers(padded));
    // (the workspace has room for two parts a warp: one is used, and two for each of 160 CTAs)
    join.cta_part = join.part + static_cast<size_t>(most_workers(padded)) * heads * (padded + 2);
    return int8 ? launch_attention_int8_groups(a, dev, join, s) : launch_attention_e4m3_groups(a, dev, join, s);
}

}  // namespace w4a16
