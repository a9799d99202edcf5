// Keys and values of requests read back from a paged cache in 8 bits with a scale
// for each group of tokens and head (w4a16_scaled_read): out = code * scale, rounded
// once.
//
// Bound by memory, mostly by its writes (two or four bytes a code).  A CTA takes a
// chunk of output rows: where each lies in the cache goes to shared memory once,
// for all heads; then a thread has one unit of 16 values of a row, two runs of eight
// so that the lanes of a head touch whole sectors, and takes it of several rows at a
// time, all their codes and scales requested before the first is used.  (CTAs that go on
// to further chunks, whose places they look up meanwhile, took 175 us for the case below:
// four CTAs an SM that come and go overlap as well, and need fewer registers.)
//
// Measured on one GB300 (copies run at 6.77 TB/s), 8 heads of 128 dims to bf16: 64 requests
// of 0 to 8192 tokens 167.5 us, 1.10 GB at 6.56 TB/s (0.97 of the copy rate); 300 tokens 3.7
// us (2.6 in a graph): launch, row, block id, codes, one after another.
#include <algorithm>

#include "common.cuh"
#include "scaled.h"
#include "scaled_core.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;   // of a CTA at most
constexpr int kBatch = 4;   // rows of a thread on their way
constexpr int kPerSm = 4;   // CTAs of an SM

struct ReadPlan {
    int chunk;       // rows of a CTA
    int range;       // units of a CTA
    uint32_t magic;  // of the cache's group
};

// Where a row's codes and scales begin (of head 0).
struct RowPlace {
    int64_t k, v, ks, vs;
};

// eight codes times their scale, to out
template <bool INT8, bool F32>
__device__ __forceinline__ void put8(const uint2& c, float scale, void* out) {
    float x[8];
    {
        float a[4], b[4];
        codes_to_f32<INT8>(c.x, a);
        codes_to_f32<INT8>(c.y, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = a[i] * scale, x[4 + i] = b[i] * scale;
    }
    if (F32) {
        float4* o = static_cast<float4*>(out);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *static_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Where the rows of a chunk lie.
struct Places {
    RowPlace at[kRows];
    int state[kRows];  // 1: a token, 0: none of its own (zeros), -1: nobody's row
};

// Looks a row up (one thread); starts: every stride-th of row_start, samples of them.
__device__ __forceinline__ int find_row(const ScaledReadArgs& a, uint32_t magic, const int* starts, int stride, int samples, int64_t row, RowPlace& at) {
    if (row < starts[0] || row >= starts[kThreads]) return -1;
    // the last b with row_start[b] <= row: among the samples, then between two of them
    int lo = 0, hi = samples;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (starts[mid] <= row) lo = mid;
        else hi = mid;
    }
    int begin = starts[lo];
    lo *= stride;
    hi = min(lo + stride, a.B);
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2, first = a.row_start[mid];
        if (first <= row) lo = mid, begin = first;
        else hi = mid;
    }
    const int b = min(lo, a.B - 1);
    const int64_t token = row - begin + (a.first ? a.first[b] : 0);
    if (token < 0 || token >= static_cast<int64_t>(a.columns) * a.cache.page) return 0;
    const unsigned col = static_cast<unsigned>(token) / static_cast<unsigned>(a.cache.page);
    const int in = static_cast<int>(token - static_cast<int64_t>(col) * a.cache.page);
    const int64_t block = a.block_table[b * a.table_stride + col];
    if (block < 0 || block >= a.cache.blocks) return 0;
    const int64_t of = magic ? __umulhi(in, magic) : in;
    at = RowPlace{block * a.cache.k_block + in * a.cache.k_token, block * a.cache.v_block + in * a.cache.v_token,
                  block * a.cache.ks_block + of * a.cache.ks_group, block * a.cache.vs_block + of * a.cache.vs_group};
    return 1;
}

template <bool INT8, bool F32>
__global__ void __launch_bounds__(kThreads, kPerSm) k_scaled_read(const ScaledReadArgs a, const ReadPlan plan) {
    __shared__ int starts[kThreads + 1];
    __shared__ Places p;
    grid_dependency_wait();
    grid_dependents_launch();
    const int stride = (a.B + kThreads) / kThreads;  // B + 1 entries, kThreads of them at most
    const int samples = a.B / stride + 1;
    if (static_cast<int>(threadIdx.x) < samples) starts[threadIdx.x] = a.row_start[threadIdx.x * stride];
    if (threadIdx.x == kThreads - 1) starts[kThreads] = a.row_start[a.B];
    __syncthreads();
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * plan.chunk;
    const int here = a.rows - r0 < plan.chunk ? static_cast<int>(a.rows - r0) : plan.chunk;
    uint32_t error = 0u;
    if (static_cast<int>(threadIdx.x) < here) {
        const int state = find_row(a, plan.magic, starts, stride, samples, r0 + threadIdx.x, p.at[threadIdx.x]);
        p.state[threadIdx.x] = state;
        if (state == 0) error = W4A16_DEVERR_SLOT;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && starts[kThreads] > a.rows) error |= W4A16_DEVERR_BLOCKS;
    if (error) raise_device_error(a.err, error);
    __syncthreads();

    const int per_head = a.cache.dim / 16, units = 2 * a.cache.heads * per_head;
    const int u0 = blockIdx.y * plan.range, range = min(plan.range, units - u0);
    const int step = kThreads / range, mine = static_cast<int>(threadIdx.x) / range;
    const bool idle = mine >= step;
    const int u = u0 + static_cast<int>(threadIdx.x) - mine * range;
    const bool value = u >= a.cache.heads * per_head;
    const int head = u / per_head - (value ? a.cache.heads : 0), at = u % per_head;
    const int d0 = at * 8, d1 = d0 + a.cache.dim / 2;
    const uint8_t* codes = static_cast<const uint8_t*>(value ? a.cache.v : a.cache.k) + head * (value ? a.cache.v_head : a.cache.k_head);
    const float* scales = (value ? a.cache.v_scale + head * a.cache.vs_head : a.cache.k_scale + head * a.cache.ks_head);
    constexpr int kSize = F32 ? 4 : 2;
    const int64_t out_row = (value ? a.v_row : a.k_row) * kSize;
    uint8_t* const out = static_cast<uint8_t*>(value ? a.v_out : a.k_out) + head * (value ? a.v_out_head : a.k_out_head) * kSize + r0 * out_row;

    if (idle) return;
    for (int from = mine; from < here; from += kBatch * step) {
        uint2 c0[kBatch], c1[kBatch];
        float f[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int row = from + j * step;
            c0[j] = c1[j] = make_uint2(0u, 0u);
            f[j] = 0.f;
            if (row >= here || p.state[row] <= 0) continue;
            const uint8_t* c = codes + (value ? p.at[row].v : p.at[row].k);
            c0[j] = *reinterpret_cast<const uint2*>(c + d0);
            c1[j] = *reinterpret_cast<const uint2*>(c + d1);
            f[j] = scales[value ? p.at[row].vs : p.at[row].ks];
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int row = from + j * step;
            if (row >= here || p.state[row] < 0) continue;
            uint8_t* o = out + row * out_row;
            put8<INT8, F32>(c0[j], f[j], o + d0 * kSize);
            put8<INT8, F32>(c1[j], f[j], o + d1 * kSize);
        }
    }
}

}  // namespace

cudaError_t launch_scaled_read(const ScaledReadArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    const int units = 2 * a.cache.heads * (a.cache.dim / 16);
    ReadPlan plan{};
    plan.magic = group_magic(a.cache.group);
    int parts = (units + kThreads - 1) / kThreads;
    plan.range = (units + parts - 1) / parts;
    parts = (units + plan.range - 1) / plan.range;
    // as many rows as a thread takes at once, up to kRows while SMs have several waves of CTAs;
    // fewer where there are not enough for all SMs
    const int step = std::max(kThreads / plan.range, 1);
    plan.chunk = std::min(kRows, step * kBatch);
    while (plan.chunk * 2 <= kRows && a.rows * parts / (plan.chunk * 2) >= 4 * kPerSm * dev.sms) plan.chunk *= 2;
    while (plan.chunk > step && a.rows * parts / plan.chunk < dev.sms) plan.chunk = std::max(step, plan.chunk / 2);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((a.rows + plan.chunk - 1) / plan.chunk), static_cast<unsigned>(parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool int8 = a.cache.dtype == W4A16_CACHE_INT8;
    const cudaError_t e = int8 ? (a.out_f32 ? cudaLaunchKernelEx(&cfg, k_scaled_read<true, true>, a, plan) : cudaLaunchKernelEx(&cfg, k_scaled_read<true, false>, a, plan))
                               : (a.out_f32 ? cudaLaunchKernelEx(&cfg, k_scaled_read<false, true>, a, plan) : cudaLaunchKernelEx(&cfg, k_scaled_read<false, false>, a, plan));
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4a16
