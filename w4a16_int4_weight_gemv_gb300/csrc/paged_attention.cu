// w4a16_paged_attention: workspace layout and choice of the kernel.
#include "paged.h"

namespace w4a16 {

// paged_attention_bf16.cu, paged_attention_e4m3.cu
cudaError_t launch_attention_bf16(const AttentionArgs& a, const DeviceInfo& dev, uint32_t* arrived, float* part, int most,
                                  cudaStream_t s);
cudaError_t launch_attention_e4m3(const AttentionArgs& a, const DeviceInfo& dev, uint32_t* arrived, float* part, int most,
                                  cudaStream_t s);

namespace {
constexpr int kMostCtas = 320;  // of a launch: two on each of 152 SMs, rounded up
constexpr size_t kCounterBytes = kMostCtas * sizeof(uint32_t);
}  // namespace

// A counter per CTA, then two partial rows per CTA: o [heads][dim], m, l.
size_t paged_attention_workspace(int q_heads, int kv_heads, int dim) {
    const int heads = q_heads / kv_heads > 8 ? 16 : 8;
    const int padded = (dim + 63) / 64 * 64;
    return kCounterBytes + static_cast<size_t>(kMostCtas) * 2 * heads * (padded + 2) * sizeof(float);
}

cudaError_t launch_paged_attention(const AttentionArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    uint32_t* arrived = static_cast<uint32_t*>(a.workspace);
    float* part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCounterBytes);
    return a.cache.dtype == W4A16_CACHE_BF16 ? launch_attention_bf16(a, dev, arrived, part, kMostCtas, s)
                                             : launch_attention_e4m3(a, dev, arrived, part, kMostCtas, s);
}

}  // namespace w4a16
