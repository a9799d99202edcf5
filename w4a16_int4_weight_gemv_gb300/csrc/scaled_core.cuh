// 8-bit codes of a w4a16_scaled_cache.  Internal to the library.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace w4a16 {
namespace {

// Four codes of a word as floats, exactly.
template <bool INT8>
__device__ __forceinline__ void codes_to_f32(uint32_t w, float (&x)[4]) {
    if (INT8) {
        // 2^23 + (code + 128), the code's byte as the float's lowest one
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | i)) - 8388736.f;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

// Four values of a code's range (|x| <= 127 or 448, a little over it by rounding
// of a rotation) to the nearest codes, ties to even.
template <bool INT8>
__device__ __forceinline__ uint32_t f32_to_codes(float x0, float x1, float x2, float x3) {
    if (INT8) {
        // 1.5 * 2^23 + x rounds to a whole number whose lowest byte is the code's
        const uint32_t a = __float_as_uint(x0 + 12582912.f), b = __float_as_uint(x1 + 12582912.f);
        const uint32_t c = __float_as_uint(x2 + 12582912.f), d = __float_as_uint(x3 + 12582912.f);
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2, x3), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

}  // namespace
}  // namespace w4a16
