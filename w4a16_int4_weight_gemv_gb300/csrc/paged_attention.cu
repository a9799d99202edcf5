// w4a16_paged_attention: workspace, the two launches, and the second of them,
// which joins the rows that several CTAs of the first one share.
//
// Parts (m, l, o) of disjoint token sets join as
//     M = max m_i,  L = sum l_i 2^(m_i - M),  O = sum o_i 2^(m_i - M),  out = O / L.
// A CTA takes some heads of one row: its threads take four dims of a head
// each, in groups that take every n-th part, so that all of a row's parts are
// requested at once; the groups are joined in shared memory.  It is launched
// while the first launch runs and waits for its end, so it costs the latency
// of two dependent reads, and nothing but that where no row was split.
#include "common.cuh"
#include "paged_attention.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int kDepth = 4;  // parts a thread requests together

struct Sum {
    float top, all;
    float4 v;
};

// adds the part (m, l, o) to s
__device__ __forceinline__ void add_part(Sum& s, float m, float l, const float4& o) {
    if (l == 0.f) return;
    const float t = fmaxf(s.top, m);
    const float f0 = s.top == t ? 1.f : exp2f(s.top - t), f1 = m == t ? 1.f : exp2f(m - t);
    s.top = t;
    s.all = s.all * f0 + l * f1;
    s.v.x = s.v.x * f0 + o.x * f1, s.v.y = s.v.y * f0 + o.y * f1;
    s.v.z = s.v.z * f0 + o.z * f1, s.v.w = s.v.w * f0 + o.w * f1;
}

// Threads (x: four dims, y: head and group of parts); grid (row, slice of its heads).
__global__ void __launch_bounds__(kThreads) k_attention_join(const AttentionArgs a, const JoinPlan j, const int log_heads) {
    __shared__ Sum sums[kThreads];
    grid_dependents_launch();
    grid_dependency_wait();
    const int4 d = __ldcg(j.joins + blockIdx.x);
    const int b = d.x, row = d.y, first = d.z, last = d.w;
    if (b < 0) return;
    const int lanes = blockDim.x, groups = blockDim.y >> log_heads, group = threadIdx.y >> log_heads;
    const int h = (blockIdx.y << log_heads) + (threadIdx.y & ((1 << log_heads) - 1)), dim = threadIdx.x * 4;
    const int64_t size = static_cast<int64_t>(j.heads) * (j.padded + 2);
    Sum s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
    for (int q = first + group; q <= last; q += groups * kDepth) {
        float m[kDepth], l[kDepth];
        float4 o[kDepth];
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            const int p = min(q + i * groups, last);
            const float* part = j.part + (static_cast<int64_t>(p) * 2 + (p == first ? 1 : 0)) * size;
            o[i] = __ldcg(reinterpret_cast<const float4*>(part + h * j.padded + dim));
            m[i] = __ldcg(part + j.heads * j.padded + h);
            l[i] = q + i * groups <= last ? __ldcg(part + j.heads * (j.padded + 1) + h) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kDepth; ++i) add_part(s, m[i], l[i], o[i]);
    }
    const int me = threadIdx.y * lanes + threadIdx.x, step = lanes << log_heads;
    sums[me] = s;
    __syncthreads();
    const int G = a.q_heads / a.cache.heads, chunks = j.rows / a.cache.heads;
    const int hk = row / chunks, head = (row - hk * chunks) * j.heads + h;  // of the group
    if (group > 0 || head >= G || dim >= a.cache.dim) return;
#pragma unroll 1
    for (int g = 1; g < groups; ++g) {
        const Sum& x = sums[me + g * step];
        add_part(s, x.top, x.all, x.v);
    }
    const bool e4m3 = a.cache.dtype == W4A16_CACHE_E4M3;
    const float f = s.all != 0.f ? (e4m3 ? a.cache.v_scale[hk] : 1.f) / s.all : 0.f;
    const uint32_t lo = f32_to_bf16_rn(s.v.x * f) | (static_cast<uint32_t>(f32_to_bf16_rn(s.v.y * f)) << 16);
    const uint32_t hi = f32_to_bf16_rn(s.v.z * f) | (static_cast<uint32_t>(f32_to_bf16_rn(s.v.w * f)) << 16);
    *reinterpret_cast<uint2*>(a.out + b * a.out_request + (hk * G + head) * a.out_head + dim) = make_uint2(lo, hi);
    if (dim == 0 && a.lse)
        a.lse[static_cast<int64_t>(b) * a.q_heads + hk * G + head] =
            s.all != 0.f ? (s.top + (log2f(s.all) - (e4m3 ? kE4m3Bias : 0.f))) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t paged_attention_workspace(int q_heads, int kv_heads, int dim) {
    const int heads = q_heads / kv_heads > 8 ? 16 : 8;
    const int padded = (dim + 63) / 64 * 64;
    return kMostAttnCtas * sizeof(int4) +
           static_cast<size_t>(kMostAttnCtas) * 2 * heads * (padded + 2) * sizeof(float);
}

cudaError_t launch_paged_attention(const AttentionArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    JoinPlan join{};
    join.joins = static_cast<int4*>(a.workspace);
    join.part = reinterpret_cast<float*>(join.joins + kMostAttnCtas);
    cudaError_t e = a.cache.dtype == W4A16_CACHE_BF16 ? launch_attention_bf16(a, dev, join, s)
                                                      : launch_attention_e4m3(a, dev, join, s);
    if (e != cudaSuccess || !join.split) return e;
    const int places = join.by_row ? a.B * join.rows : join.ctas;
    // few rows: their heads over several CTAs, down to one head each
    const int lanes = join.padded / 4;
    int log_heads = join.heads == 16 ? 4 : 3;
    while (log_heads > 0 && ((lanes << log_heads) > kThreads || places * (join.heads >> log_heads) < dev.sms)) --log_heads;
    const int groups = kThreads / (lanes << log_heads);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(places, join.heads >> log_heads);
    cfg.blockDim = dim3(lanes, groups << log_heads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_attention_join, a, join, log_heads);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4a16
