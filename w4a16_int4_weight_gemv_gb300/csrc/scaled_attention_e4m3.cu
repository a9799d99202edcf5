// Attention over an e4m3 cache with scales by group.
#include "paged_attention_mma.cuh"

namespace w4a16 {

cudaError_t launch_attention_e4m3_groups(const ScaledAttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s) {
    return launch_attention_type<kE4m3Groups>(a, dev, join, s);
}

}  // namespace w4a16
