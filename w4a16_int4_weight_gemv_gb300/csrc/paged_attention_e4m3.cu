// One-token attention over an e4m3 cache.
#include "paged_attention_mma.cuh"

namespace w4a16 {

cudaError_t launch_attention_e4m3(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s) {
    return launch_attention_type<kE4m3>(a, dev, join, s);
}

}  // namespace w4a16
