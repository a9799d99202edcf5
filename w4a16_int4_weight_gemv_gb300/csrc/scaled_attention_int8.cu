// Attention over an int8 cache with scales by group.
#include "paged_attention_mma.cuh"

namespace w4a16 {

cudaError_t launch_attention_int8_groups(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s) {
    return launch_attention_type<kInt8Groups>(a, dev, join, s);
}

}  // namespace w4a16
