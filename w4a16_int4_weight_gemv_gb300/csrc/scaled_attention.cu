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
    join.part = reinterpret_cast<float*>(join.joins + most_workers(padded_dim(a.cache.dim)));
    return int8 ? launch_attention_int8_groups(a, dev, join, s) : launch_attention_e4m3_groups(a, dev, join, s);
}

}  // namespace w4a16
