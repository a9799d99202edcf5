// Rotary positions with several axes, and the append of keys and values to
// the paged cache (w4a16_rope_append).
//
// A pair (x1, x2) of a head is a complex number turned by e^(i a), a = pos *
// f.  The angle is formed in half turns, pos * (f / pi), as an unevaluated
// sum of two floats (f / pi to 48 bits, the product's rounding error by one
// fused multiply-add), its high part reduced modulo 2 exactly, and sincospif
// takes the rest (positions of 2^24 and more, and negative ones, go through
// 64 bits): the turn is good to about 2^-21 whatever the position, where the
// rounded product pos * f alone is off by up to pos * f * 2^-24 radians.
//
// Bound by memory: every value is read once and written once.  A CTA takes
// groups of tokens: it forms the cosines and sines of their pairs in shared
// memory once, for all heads.  A thread has one unit of 16 values of a token,
// two runs of eight so that the lanes of a head touch whole sectors, and takes
// it of TOKENS tokens of a group.  The next group's values, slots and positions
// are requested before this one's are turned and written: reads and writes
// overlap within a CTA, and two buffers of angles leave one barrier a group.
//
// Measured on one GB300 (copies run at 6.67 TB/s) in a CUDA graph, 32 query and 8
// key/value heads of 128: 16384 tokens of three axes into bf16 62.3 us (6.47 TB/s),
// 4095 tokens into e4m3 18.1 us (5.09 TB/s; 65 % of the issue slots over the whole
// call, with 39 % of the warps an SM could hold: what limits it is not shown), one
// token 1.5 us.  With a group's requests after the last one's writes: 66.6, 20.2 and
// 1.9 us.  More CTAs an SM leave too few registers: one token a thread and five CTAs
// 88 us for the first.  (As it is, 16 bytes a thread are spilled with one token a
// thread, 24 with two.)
#include <algorithm>

#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"
#include "rope_core.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;  // at most
constexpr int kAngles = 2048;  // of a group at most: tokens times pairs
constexpr int kMany = 2;       // tokens of a thread and group where there are many:
constexpr int kOften = 16;     // groups of an SM at least
// CTAs of kThreads threads an SM: 64 registers each, 80 with several tokens on their way
constexpr int per_sm(int tokens) { return tokens == 1 ? 4 : 3; }

// Scales whose reciprocal, remainders and bound stay in a float's range.
__device__ __forceinline__ bool ordinary(float scale) { return fabsf(scale) >= 0x1p-100f && fabsf(scale) <= 0x1p100f; }

// Eight values over the scale as e4m3, saturating (a NaN stays one).  DIVIDE: by
// divisions, for any scale (one of 0: infinities and NaN).  Else, for ordinary
// scales, x times the reciprocal, corrected by its remainder, which rounds as a
// division does; two at a time (f32x2).  With the bound as one instruction that
// takes 0.35 us off the 18.5 of 4095 tokens.  There t = -x within the bound (the
// sign of -scale on it) and the reciprocal is negative: so a remainder of 0 leaves
// the sign of a quotient of 0 as it is.
template <bool DIVIDE>
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
    const float size = fabsf(scale), inv = -1.f / size, most = -480.f * scale;  // 464 and more round to 448
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[2];
        if (DIVIDE) {
            v[0] = x[2 * i] / scale, v[1] = x[2 * i + 1] / scale;
        } else {
            float t[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(t[e]) : "f"(x[2 * i + e]), "f"(most));
            asm("{.reg .b64 t, q, r, s, n;\n mov.b64 t, {%2, %3};\n mov.b64 n, {%4, %4};\n mov.b64 s, {%5, %5};\n"
                "mul.rn.f32x2 q, t, n;\n fma.rn.f32x2 r, q, s, t;\n fma.rn.f32x2 r, r, n, q;\n mov.b64 {%0, %1}, r;}"
                : "=f"(v[0]), "=f"(v[1]) : "f"(t[0]), "f"(t[1]), "f"(inv), "f"(size));
        }
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Units of a token: dim / 16 of each head, query heads first, then key heads,
// then value heads.  Unit u of a head holds the values d0 .. d0 + 7 and
// d1 .. d1 + 7; the first rotary / 16 units are turned.  grid: (groups of
// `group` tokens, ranges of `range` units of a token).
// The angles of a unit's eight pairs lie in four float4 (cos, sin, cos, sin), the
// i-th of all units of a token next to one another: no two lanes of a head meet
// in a bank.
template <int TOKENS>
__global__ void __launch_bounds__(kThreads, per_sm(TOKENS)) k_rope_append(const RopeArgs a, const int group, const int range) {
    extern __shared__ __align__(16) float4 angles[];  // [2][group * half / 2]
    const int per_head = a.dim / 16, half = a.rotary / 2, turned = half / 8;  // turned: units of a head
    const int step = group / TOKENS;  // tokens of a group that the threads take at once
    const int units = (a.q_heads + 2 * a.cache.heads) * per_head;
    const int u_begin = blockIdx.y * range, u_count = min(range, units - u_begin);
    // this thread's unit: of which token of the group, head and dims
    const int my_token = static_cast<int>(threadIdx.x) / u_count;
    int head, kind, d0, d1;
    bool halves = false, neighbours = false;
    {
        const int u = u_begin + static_cast<int>(threadIdx.x) - my_token * u_count;
        head = u / per_head;
        const int at = u - head * per_head;
        kind = head < a.q_heads ? 0 : head < a.q_heads + a.cache.heads ? 1 : 2;  // query, key, value
        head -= kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + a.cache.heads;
        neighbours = kind != 2 && a.interleaved;
        halves = kind != 2 && !a.interleaved && at < turned;
        if (halves) {
            d0 = at * 8;
            d1 = d0 + half;
        } else {  // the two halves of what is turned in place or not at all
            const int from = kind != 2 && !a.interleaved ? a.rotary : 0;
            d0 = from + (at - from / 16) * 8;
            d1 = d0 + (a.dim - from) / 2;
        }
    }
    const uint16_t* src = kind == 0 ? a.q + head * a.q_head : kind == 1 ? a.k + head * a.k_head : a.v + head * a.v_head;
    const int64_t src_token = kind == 0 ? a.q_token : kind == 1 ? a.k_token : a.v_token;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * group;
    // the pair whose angle this thread forms first of every group (further ones: in `turns`)
    const int first_token = half ? static_cast<int>(threadIdx.x) / half : 0;
    const int first_pair = static_cast<int>(threadIdx.x) - first_token * half;
    float first_freq = 0.f;
    const int* first_pos = a.positions;
    if (first_token < group && half) {
        int axis = 0;
        while (axis < 3 && first_pair >= a.axis_end[axis]) ++axis;
        first_pos += axis * a.axis_stride + first_token;
    }
    const int page_shift = (a.cache.page & (a.cache.page - 1)) == 0 ? 31 - __clz(a.cache.page) : -1;
    bool bad = false;
    int buffer = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    if (first_token < group && half) first_freq = a.inv_freq[first_pair];

    const auto load = [&](int64_t t0, uint4 (&v0)[TOKENS], uint4 (&v1)[TOKENS], int (&slot)[TOKENS], int& pos) {
        const int tokens = a.T - t0 < group ? static_cast<int>(a.T - t0) : group;
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) {
            const int token = my_token + j * step;
            slot[j] = -1;
            if (my_token >= step || token >= tokens) continue;
            const uint16_t* x = src + (t0 + token) * src_token;
            slot[j] = kind ? a.slots[t0 + token] : 0;
            v0[j] = *reinterpret_cast<const uint4*>(x + d0);
            v1[j] = *reinterpret_cast<const uint4*>(x + d1);
        }
        if (half && first_token < tokens) pos = first_pos[t0];
    };
    const auto put = [&](float4* cs, int token, int pair, int pos, float f) {
        float2 c = turn_of(pos, f);
        if (a.inverse) c.y = -c.y;
        cs += token * 4 * turned;
        cs += a.interleaved ? (pair & 3) / 2 * 2 * turned + pair / 4 : (pair & 7) / 2 * turned + pair / 8;
        reinterpret_cast<float2*>(cs)[pair & 1] = c;
    };
    const auto turns = [&](int64_t t0, int pos) {
        float4* const cs = angles + buffer * (group * half / 2);
        const int tokens = a.T - t0 < group ? static_cast<int>(a.T - t0) : group;
        if (half && first_token < tokens) put(cs, first_token, first_pair, pos, first_freq);
        for (int i = threadIdx.x + blockDim.x; i < tokens * half; i += blockDim.x) {
            const int token = i / half, pair = i - token * half;
            int axis = 0;
            while (axis < 3 && pair >= a.axis_end[axis]) ++axis;
            put(cs, token, pair, a.positions[axis * a.axis_stride + t0 + token], a.inv_freq[pair]);
        }
    };

    int64_t t0 = static_cast<int64_t>(blockIdx.x) * group;
    uint4 v0[TOKENS], v1[TOKENS];
    int slot[TOKENS], pos = 0;
    load(t0, v0, v1, slot, pos);
    turns(t0, pos);
    __syncthreads();
    while (true) {
        const bool more = a.T - t0 > stride;
        uint4 n0[TOKENS], n1[TOKENS];
        int nslot[TOKENS];
        if (more) load(t0 + stride, n0, n1, nslot, pos);
        const float4* const cs = angles + buffer * (group * half / 2);
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) {
            const int token = my_token + j * step, to = slot[j];
            if (to == -1) continue;
            if (kind && (to < 0 || to >= a.cache.blocks * a.cache.page)) {
                bad = true;
                continue;
            }
            float p[8], q[8];
            unpack8(v0[j], p);
            unpack8(v1[j], q);
            if (halves) {
                const float4* c = cs + token * 4 * turned + d0 / 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 e = c[i * turned];
                    const float y0 = p[2 * i] * e.x - q[2 * i] * e.y, y1 = p[2 * i + 1] * e.z - q[2 * i + 1] * e.w;
                    q[2 * i] = q[2 * i] * e.x + p[2 * i] * e.y;
                    q[2 * i + 1] = q[2 * i + 1] * e.z + p[2 * i + 1] * e.w;
                    p[2 * i] = y0, p[2 * i + 1] = y1;
                }
            } else if (neighbours) {
                if (d0 < a.rotary) turn_neighbours(p, cs + token * 4 * turned + d0 / 8, 2 * turned);
                if (d1 < a.rotary) turn_neighbours(q, cs + token * 4 * turned + d1 / 8, 2 * turned);
            }
            if (kind == 0) {
                uint16_t* dst = a.q_out + (t0 + token) * a.qo_token + head * a.qo_head;
                *reinterpret_cast<uint4*>(dst + d0) = pack8(p);
                *reinterpret_cast<uint4*>(dst + d1) = pack8(q);
                continue;
            }
            const int64_t block = page_shift >= 0 ? static_cast<unsigned>(to) >> page_shift : static_cast<unsigned>(to) / static_cast<unsigned>(a.cache.page);
            const int64_t place = to - block * a.cache.page;
            const int64_t offset = kind == 1 ? block * a.cache.k_block + place * a.cache.k_token + head * a.cache.k_head
                                             : block * a.cache.v_block + place * a.cache.v_token + head * a.cache.v_head;
            void* cache = kind == 1 ? a.cache.k : a.cache.v;
            if (TOKENS > 1 || a.cache.dtype == W4A16_CACHE_BF16) {  // several tokens: never over e4m3
                uint16_t* dst = static_cast<uint16_t*>(cache) + offset;
                *reinterpret_cast<uint4*>(dst + d0) = pack8(p);
                *reinterpret_cast<uint4*>(dst + d1) = pack8(q);
            } else {
                const float scale = kind == 1 ? a.cache.k_scale[head] : a.cache.v_scale[head];
                uint8_t* dst = static_cast<uint8_t*>(cache) + offset;
                if (!ordinary(scale)) {
                    *reinterpret_cast<uint2*>(dst + d0) = pack8_e4m3<true>(p, scale);
                    *reinterpret_cast<uint2*>(dst + d1) = pack8_e4m3<true>(q, scale);
                } else {
                    *reinterpret_cast<uint2*>(dst + d0) = pack8_e4m3<false>(p, scale);
                    *reinterpret_cast<uint2*>(dst + d1) = pack8_e4m3<false>(q, scale);
                }
            }
        }
        if (!more) break;
        t0 += stride;
        buffer ^= 1;
        turns(t0, pos);
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) v0[j] = n0[j], v1[j] = n1[j], slot[j] = nslot[j];
        __syncthreads();
    }
    if (bad) raise_device_error(a.err, W4A16_DEVERR_SLOT);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    const int units = (a.q_heads + 2 * a.cache.heads) * (a.dim / 16), half = a.rotary / 2;
    // a token's units over as few CTAs as hold them, over more where tokens are few
    int parts = (units + kThreads - 1) / kThreads;
    while (parts < 16 && units / parts > 64 && a.T * parts < dev.sms) parts *= 2;
    const int range = (units + parts - 1) / parts;
    parts = (units + range - 1) / range;
    // tokens that the threads take at once: but a CTA for every SM at least
    int64_t step = std::max(kThreads / range, 1);
    if (half) step = std::min<int64_t>(step, kAngles / (kMany * half));
    step = std::max<int64_t>(1, std::min<int64_t>(step, a.T * parts / dev.sms));
    const int threads = static_cast<int>(step * range + 31) / 32 * 32;
    // and how often: several times over bf16 where that leaves enough groups for the SMs to
    // end together (4095 tokens of 32 + 2 * 8 heads of 128: 18.3 us against 18.9, 16384 63
    // against 67; 1500 tokens 8.6 against 7.8; over e4m3, where fewer registers are free, 4095
    // tokens 20.0 against 18.8)
    const bool bf16 = a.cache.heads == 0 || a.cache.dtype == W4A16_CACHE_BF16;
    const bool many = bf16 && a.T * parts >= step * kMany * kOften * dev.sms;
    const int group = static_cast<int>(step) * (many ? kMany : 1);
    const int smem = group * half * 16;
    auto* kernel = many ? k_rope_append<kMany> : k_rope_append<1>;
    const cudaError_t rc = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (rc != cudaSuccess) return rc;
    int64_t ctas = (a.T + group - 1) / group;
    const int64_t wave = std::max<int64_t>(1, static_cast<int64_t>(per_sm(many ? kMany : 1) * kThreads / threads) * dev.sms / parts);
    if (ctas > wave) ctas = wave;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(parts));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, group, range);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4a16
