// One-token attention over a bf16 cache.
#include "paged_attention_mma.cuh"

namespace w4a16 {

cudaError_t launch_attention_bf16(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s) {
    return launch_attention_type<false>(a, dev, join, s);
}

}  // namespace w4a16
