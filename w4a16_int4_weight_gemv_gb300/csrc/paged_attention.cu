// Attention of one new token per request over a paged key/value cache
// (w4a16_paged_attention).
//
// One CTA per request and query head.  Its eight warps take the visible
// tokens in turn, each keeping the running maximum m, the sum l of
// exp(s - m) and the weighted sum o of values of its own tokens in fp32
// (a new maximum m' scales l and o by exp(m - m')); at the end the warps'
// triples are joined in shared memory in the same way.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"

namespace w4a16 {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxDim = 256;

__device__ __forceinline__ float cache_value(const void* p, int64_t at, int dtype) {
    if (dtype == W4A16_CACHE_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[at], __NV_E4M3);
    return __half2float(__half(h));
}

__global__ void __launch_bounds__(kWarps * 32) k_paged_attention(const AttentionArgs a) {
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][kMaxDim];
    const int b = blockIdx.x / a.q_heads, h = blockIdx.x - b * a.q_heads;
    const int hk = h / (a.q_heads / a.cache.heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.cache.dim;
    uint32_t bad = 0u;
    int64_t len = a.kv_len[b];
    if (len < 0) {
        bad = W4A16_DEVERR_SLOT;
        len = 0;
    }
    const int64_t most = static_cast<int64_t>(a.columns) * a.cache.page;
    if (len > most) {
        bad = W4A16_DEVERR_SLOT;
        len = most;
    }
    const int64_t start = a.window > 0 && len > a.window ? len - a.window : 0;
    const bool e4m3 = a.cache.dtype == W4A16_CACHE_E4M3;
    const float scale = a.scale * (e4m3 ? a.cache.k_scale[hk] : 1.f);
    float q[8], o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < D ? bf16_to_f32(a.q[b * a.q_request + h * a.q_head + d]) : 0.f;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int64_t t = start + warp; t < len; t += kWarps) {
        const int64_t col = t / a.cache.page, place = t - col * a.cache.page;
        const int64_t id = a.block_table[b * a.table_stride + col];
        if (id < 0 || id >= a.cache.blocks) {
            bad = W4A16_DEVERR_SLOT;
            continue;
        }
        const int64_t kat = id * a.cache.k_block + place * a.cache.k_token + hk * a.cache.k_head;
        const int64_t vat = id * a.cache.v_block + place * a.cache.v_token + hk * a.cache.v_head;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < D) s = fmaf(q[i], cache_value(a.cache.k, kat + lane + 32 * i, a.cache.dtype), s);
#pragma unroll
        for (int d = 16; d; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        s *= scale;
        const float top = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.f : expf(m - top);
        const float p = s == -INFINITY ? 0.f : expf(s - top);
        m = top;
        l = l * keep + p;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < D)
                o[i] = fmaf(p, cache_value(a.cache.v, vat + lane + 32 * i, a.cache.dtype), o[i] * keep);
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sm_o[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w]);
    for (int w = 0; w < kWarps; ++w) sum += sm_l[w] != 0.f ? sm_l[w] * expf(sm_m[w] - top) : 0.f;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w)
            if (sm_l[w] != 0.f) v = fmaf(sm_o[w][d], expf(sm_m[w] - top), v);
        v = sum != 0.f ? v / sum * (e4m3 ? a.cache.v_scale[hk] : 1.f) : 0.f;
        a.out[b * a.out_request + h * a.out_head + d] = f32_to_bf16_rn(v);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[static_cast<int64_t>(b) * a.q_heads + h] = sum != 0.f ? top + logf(sum) : -INFINITY;
    if (bad && lane == 0) raise_device_error(a.err, bad);
}

}  // namespace

size_t paged_attention_workspace(int q_heads, int kv_heads, int dim) {
    (void)q_heads, (void)kv_heads, (void)dim;
    return 16;
}

cudaError_t launch_paged_attention(const AttentionArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    (void)dev;
    k_paged_attention<<<a.B * a.q_heads, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace w4a16
