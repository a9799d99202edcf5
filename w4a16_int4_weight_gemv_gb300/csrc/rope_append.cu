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
// Bound by memory: every value is read once and written once.  A CTA serves
// one token at a time: its first threads form the cosines and sines of all
// pairs in shared memory, which every head of the token then reads.  A thread
// moves units of 16 values (two 16-byte loads), loaded before the angles are
// formed.
#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 128;

// the high and low parts of 1 / pi
constexpr float kInvPiHi = 0.31830987334251404f;
constexpr float kInvPiLo = 1.2841276486597053e-08f;

// cos and sin of pos * f
__device__ __forceinline__ float2 turn_of(int pos, float f) {
    float r;
    if (static_cast<unsigned>(pos) < (1u << 24)) {
        const float gh = f * kInvPiHi;
        const float gl = fmaf(f, kInvPiLo, fmaf(f, kInvPiHi, -gh));
        const float p = static_cast<float>(pos);  // exact
        const float th = p * gh;
        r = (th - 2.f * rintf(0.5f * th)) + fmaf(p, gl, fmaf(p, gh, -th));  // the difference is exact
    } else {  // a position no float holds (or a negative one): 53 bits of the half turns
        const double t = static_cast<double>(pos) * (static_cast<double>(f) * 0.31830988618379067154);
        r = static_cast<float>(t - 2.0 * rint(0.5 * t));
    }
    float2 cs;
    sincospif(r, &cs.y, &cs.x);
    return cs;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
        x[2 * i + 1] = bf16_to_f32(w[i] >> 16);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = f32_to_bf16_rn(x[2 * i]) | (static_cast<uint32_t>(f32_to_bf16_rn(x[2 * i + 1])) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// eight values over the scale as e4m3, saturating (a NaN stays one)
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] / scale, x[2 * i + 1] / scale), __NV_SATFINITE,
                                        __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Units of a token: dim / 16 of each head, query heads first, then key heads,
// then value heads.  Unit u of a head holds the values d0 .. d0 + 7 and
// d1 .. d1 + 7; the first rotary / 16 units are turned.
__global__ void __launch_bounds__(kThreads) k_rope_append(const RopeArgs a) {
    __shared__ float2 cs[kMaxPairs];
    const int per_head = a.dim / 16, half = a.rotary / 2;
    const int units = (a.q_heads + 2 * a.cache.heads) * per_head;
    const int parts = gridDim.y;
    uint32_t bad = 0u;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        for (int i = threadIdx.x; i < half; i += kThreads) {
            int axis = 0;
            while (axis < 3 && i >= a.axis_end[axis]) ++axis;
            float2 v = turn_of(a.positions[axis * a.axis_stride + t], a.inv_freq[i]);
            if (a.inverse) v.y = -v.y;
            cs[i] = v;
        }
        __syncthreads();
        int64_t slot = -1;
        if (a.cache.heads) {
            slot = a.slots[t];
            if (slot != -1 && (slot < 0 || slot >= a.cache.blocks * a.cache.page)) {
                bad = W4A16_DEVERR_SLOT;
                slot = -1;
            }
        }
        const int64_t block = slot < 0 ? 0 : slot / a.cache.page;
        const int64_t place = slot < 0 ? 0 : slot - block * a.cache.page;
        for (int u = blockIdx.y * kThreads + threadIdx.x; u < units; u += parts * kThreads) {
            int head = u / per_head;
            const int unit = u - head * per_head;
            const bool turned = unit * 16 < a.rotary;
            const bool halves = turned && !a.interleaved;
            const int d0 = halves ? unit * 8 : unit * 16;
            const int d1 = halves ? d0 + half : d0 + 8;
            const uint16_t* src;
            int kind = 0;  // query, key, value
            if (head < a.q_heads) {
                src = a.q + t * a.q_token + head * a.q_head;
            } else {
                if (slot < 0) continue;
                head -= a.q_heads;
                kind = head < a.cache.heads ? 1 : 2;
                if (kind == 2) head -= a.cache.heads;
                src = kind == 1 ? a.k + t * a.k_token + head * a.k_head
                                : a.v + t * a.v_token + head * a.v_head;
            }
            const uint4 v0 = *reinterpret_cast<const uint4*>(src + d0);
            const uint4 v1 = *reinterpret_cast<const uint4*>(src + d1);
            float x[8], y[8];
            unpack8(v0, x);
            unpack8(v1, y);
            if (turned && kind != 2) {
                if (halves) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 c = cs[d0 + i];
                        const float p = x[i] * c.x - y[i] * c.y, q = y[i] * c.x + x[i] * c.y;
                        x[i] = p;
                        y[i] = q;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 c = cs[d0 / 2 + i], e = cs[d0 / 2 + 4 + i];
                        const float p = x[2 * i] * c.x - x[2 * i + 1] * c.y;
                        x[2 * i + 1] = x[2 * i + 1] * c.x + x[2 * i] * c.y;
                        x[2 * i] = p;
                        const float q = y[2 * i] * e.x - y[2 * i + 1] * e.y;
                        y[2 * i + 1] = y[2 * i + 1] * e.x + y[2 * i] * e.y;
                        y[2 * i] = q;
                    }
                }
            }
            if (kind == 0) {
                uint16_t* dst = a.q_out + t * a.qo_token + head * a.qo_head;
                *reinterpret_cast<uint4*>(dst + d0) = pack8(x);
                *reinterpret_cast<uint4*>(dst + d1) = pack8(y);
                continue;
            }
            const int64_t at = kind == 1 ? block * a.cache.k_block + place * a.cache.k_token + head * a.cache.k_head
                                         : block * a.cache.v_block + place * a.cache.v_token + head * a.cache.v_head;
            void* cache = kind == 1 ? a.cache.k : a.cache.v;
            if (a.cache.dtype == W4A16_CACHE_BF16) {
                uint16_t* dst = static_cast<uint16_t*>(cache) + at;
                *reinterpret_cast<uint4*>(dst + d0) = pack8(x);
                *reinterpret_cast<uint4*>(dst + d1) = pack8(y);
            } else {
                const float scale = kind == 1 ? a.cache.k_scale[head] : a.cache.v_scale[head];
                uint8_t* dst = static_cast<uint8_t*>(cache) + at;
                *reinterpret_cast<uint2*>(dst + d0) = pack8_e4m3(x, scale);
                *reinterpret_cast<uint2*>(dst + d1) = pack8_e4m3(y, scale);
            }
        }
        __syncthreads();
    }
    if (bad) raise_device_error(a.err, bad);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    const int units = (a.q_heads + 2 * a.cache.heads) * (a.dim / 16);
    int64_t ctas = a.T;
    const int64_t most = 16LL * dev.sms;
    if (ctas > most) ctas = most;
    // few tokens: a token's units over several CTAs, each forming the angles itself
    int parts = 1;
    const int want = (units + kThreads - 1) / kThreads;
    while (parts < want && ctas * (parts + 1) <= most) ++parts;
    k_rope_append<<<dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(parts)), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace w4a16
