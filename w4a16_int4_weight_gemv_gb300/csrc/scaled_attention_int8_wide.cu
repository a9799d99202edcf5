// Attention over an int8 cache with scales by group, 24 or 32 columns together.
#include "paged_attention_mma.cuh"

namespace w4a16 {

cudaError_t launch_attention_int8_groups_wide(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s) {
    return launch_attention_wide<kInt8Groups>(a, dev, join, s);
}

}  // namespace w4a16
