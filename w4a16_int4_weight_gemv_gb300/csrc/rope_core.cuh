// What the kernels that turn heads share (w4a16_rope_append, w4a16_scaled_append).
// Internal to the library.
#pragma once

#include "common.cuh"

namespace w4a16 {
namespace {

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
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// four neighbouring pairs; their angles: c[0] and c[step]
__device__ __forceinline__ void turn_neighbours(float (&x)[8], const float4* c, int step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 e = c[i * step];
        const float y0 = x[4 * i] * e.x - x[4 * i + 1] * e.y, y1 = x[4 * i + 2] * e.z - x[4 * i + 3] * e.w;
        x[4 * i + 1] = x[4 * i + 1] * e.x + x[4 * i] * e.y;
        x[4 * i + 3] = x[4 * i + 3] * e.z + x[4 * i + 2] * e.w;
        x[4 * i] = y0, x[4 * i + 2] = y1;
    }
}

}  // namespace
}  // namespace w4a16
