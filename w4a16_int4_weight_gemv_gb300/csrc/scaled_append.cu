// Rotary positions, and the append of keys and values to a paged cache in 8
// bits whose scales are found on the way (w4a16_scaled_append).
//
// For each group of `group` tokens and head: S = the smallest power of two with
// |value| <= most * S for the new values (and no smaller than the scale so far),
// code = value / S to the nearest.  Two properties of that S carry the kernel:
//   - the length of a pair does not change as it is turned, so S takes the
//     values as they were read: the search for it needs no angle and waits for none;
//   - x / S is x times a power of two, exact, so that codes do not depend on how
//     the quotient is formed, and growing the scale shifts the codes that are there.
// With M the largest magnitude as it was read, S is 2^e(M) or, where the length of
// some pair passes most * 2^e(M), twice that: one integer maximum over the bits,
// then a comparison of squares scaled into a float's range.
//
// A CTA has the runs (new tokens of one group) that begin in its chunk of tokens,
// and a warp one run of one key or value head at a time: values in registers,
// their maximum by one reduction, old codes shifted where the scale grew, new
// codes written.  Nobody else touches that run's codes and scale.  Queries are
// turned by CTAs of their own in the same launch.
#include <algorithm>

#include "common.cuh"
#include "rope_core.cuh"
#include "scaled.h"
#include "scaled_core.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 32;  // tokens of a CTA at most
constexpr int kKeep = 4;    // steps of a run whose values stay in registers

struct AppendPlan {
    int chunk;                // tokens of a CTA
    int kv_parts, items;      // CTAs of a chunk for keys and values, heads (key, then value) of each
    int range;                // units of a query CTA
    uint32_t unit_magic;      // unit / (dim / 16) = unit * unit_magic >> 16
    uint32_t magic;           // of the cache's group
};

// The smallest e with x <= most * 2^e, of positive x (bits), from -126 on.
template <bool INT8>
__device__ __forceinline__ int exponent_for(uint32_t bits) {
    // most = 1.75 * 2^8 (e4m3) or 1.984375 * 2^6 (int8)
    const int e = static_cast<int>(bits >> 23) - 127 - (INT8 ? 6 : 8) + ((bits & 0x7FFFFFu) > (INT8 ? 0x7E0000u : 0x600000u) ? 1 : 0);
    return max(e, -126);
}

// Where unit `at` of a head has its two runs of eight values.
struct Place {
    int d0, d1;
    bool halves, neighbours;
};
__device__ __forceinline__ Place place_of(int at, int dim, int rotary, bool turn, bool interleaved) {
    Place p;
    p.halves = turn && !interleaved && at < rotary / 16;
    p.neighbours = turn && interleaved;
    if (p.halves) {
        p.d0 = at * 8;
        p.d1 = p.d0 + rotary / 2;
    } else {
        const int from = turn && !interleaved ? rotary : 0;
        p.d0 = from + (at - from / 16) * 8;
        p.d1 = p.d0 + (dim - from) / 2;
    }
    return p;
}

__device__ __forceinline__ void turn(float (&p)[8], float (&q)[8], const Place& at, const float4* cs, int rotary) {
    const int turned = rotary / 16;
    if (at.halves) {
        const float4* c = cs + at.d0 / 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 e = c[i * turned];
            const float y0 = p[2 * i] * e.x - q[2 * i] * e.y, y1 = p[2 * i + 1] * e.z - q[2 * i + 1] * e.w;
            q[2 * i] = q[2 * i] * e.x + p[2 * i] * e.y;
            q[2 * i + 1] = q[2 * i + 1] * e.z + p[2 * i + 1] * e.w;
            p[2 * i] = y0, p[2 * i + 1] = y1;
        }
    } else if (at.neighbours) {
        if (at.d0 < rotary) turn_neighbours(p, cs + at.d0 / 8, 2 * turned);
        if (at.d1 < rotary) turn_neighbours(q, cs + at.d1 / 8, 2 * turned);
    }
}

// The angles of `tokens` tokens from t0 on: the i-th float4 (cos, sin, cos, sin) of all
// units of a token next to one another.
__device__ __forceinline__ void angles_of(const ScaledAppendArgs& a, int64_t t0, int tokens, float4* angles) {
    const int half = a.rotary / 2, turned = a.rotary / 16;
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int token = i / half, pair = i - token * half;
        int axis = 0;
        while (axis < 3 && pair >= a.axis_end[axis]) ++axis;
        const float2 c = turn_of(a.positions[axis * a.axis_stride + t0 + token], a.inv_freq[pair]);
        float4* cs = angles + token * 4 * turned;
        cs += a.interleaved ? (pair & 3) / 2 * 2 * turned + pair / 4 : (pair & 7) / 2 * turned + pair / 8;
        reinterpret_cast<float2*>(cs)[pair & 1] = c;
    }
}

__device__ __forceinline__ uint32_t largest(uint32_t m, const uint4& v) {
    m = __vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
    return __vmaxu2(m, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}

// Whether the length of a pair (values times inv) passes the code range.
__device__ __forceinline__ bool longer(const uint4& v0, const uint4& v1, const Place& at, int rotary, float inv, float most2) {
    float p[8], q[8];
    unpack8(v0, p);
    unpack8(v1, q);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] *= inv, q[i] *= inv;
    if (at.halves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaf(p[i], p[i], q[i] * q[i]));  // (the squares are exact)
    } else if (at.neighbours) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (at.d0 < rotary) top = fmaxf(top, fmaf(p[i], p[i], p[i + 1] * p[i + 1]));
            if (at.d1 < rotary) top = fmaxf(top, fmaf(q[i], q[i], q[i + 1] * q[i + 1]));
        }
    }
    return top > most2;
}

template <bool INT8>
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float inv) {
    return make_uint2(f32_to_codes<INT8>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      f32_to_codes<INT8>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// Sixteen codes times ratio, to the nearest.
template <bool INT8>
__device__ __forceinline__ uint4 again(const uint4& v, float ratio) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[4];
        codes_to_f32<INT8>(w[i], x);
        w[i] = f32_to_codes<INT8>(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool INT8>
__global__ void __launch_bounds__(kThreads, 2) k_scaled_append(const ScaledAppendArgs a, const AppendPlan plan) {
    extern __shared__ __align__(16) float4 angles[];
    __shared__ int slot[kChunk + kMostGroup + 1];  // of the token before the chunk, then from its first on
    __shared__ int2 run[kChunk];                   // first token (of the chunk) and tokens
    __shared__ int runs, run_end;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_head = a.dim / 16, turned = a.rotary / 16;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * plan.chunk;
    const int64_t left = a.T - t0;
    const int here = left < plan.chunk ? static_cast<int>(left) : plan.chunk;
    grid_dependency_wait();
    grid_dependents_launch();

    if (static_cast<int>(blockIdx.y) >= plan.kv_parts) {
        // --- queries -----------------------------------------------------------
        const int u0 = (blockIdx.y - plan.kv_parts) * plan.range, range = min(plan.range, a.q_heads * per_head - u0);
        const int step = kThreads / range, mine = static_cast<int>(threadIdx.x) / range;
        const int u = u0 + static_cast<int>(threadIdx.x) - mine * range, head = u / per_head;
        const Place at = place_of(u - head * per_head, a.dim, a.rotary, a.rotary > 0, a.interleaved);
        const uint16_t* src = a.q + t0 * a.q_token + head * a.q_head;
        uint16_t* dst = a.q_out + t0 * a.qo_token + head * a.qo_head;
        constexpr int kBatch = 4;
        uint4 v0[kBatch], v1[kBatch];
        const auto load = [&](int from) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int token = from + j * step;
                if (token >= here) continue;
                v0[j] = *reinterpret_cast<const uint4*>(src + token * a.q_token + at.d0);
                v1[j] = *reinterpret_cast<const uint4*>(src + token * a.q_token + at.d1);
            }
        };
        if (mine < step) load(mine);
        angles_of(a, t0, here, angles);
        __syncthreads();
        if (mine >= step) return;
        for (int from = mine; from < here; from += kBatch * step) {
            if (from != mine) load(from);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int token = from + j * step;
                if (token >= here) continue;
                float p[8], q[8];
                unpack8(v0[j], p);
                unpack8(v1[j], q);
                turn(p, q, at, angles + token * 4 * turned, a.rotary);
                *reinterpret_cast<uint4*>(dst + token * a.qo_token + at.d0) = pack8(p);
                *reinterpret_cast<uint4*>(dst + token * a.qo_token + at.d1) = pack8(q);
            }
        }
        return;
    }

    // --- the runs that begin in the chunk ---------------------------------------
    const int group = a.cache.group;
    {
        const int most = plan.chunk + group - 1, known = left < most ? static_cast<int>(left) : most;
        for (int i = threadIdx.x; i <= known; i += kThreads) slot[i] = i || t0 ? a.slots[t0 + i - 1] : -1;
        __syncthreads();
        if (warp == 0) {
            const int s = lane < here ? slot[1 + lane] : -1, before = lane < here ? slot[lane] : -1;
            const bool valid = s >= 0 && s < a.cache.blocks * a.cache.page;
            const int place = valid ? s % group : 0;
            const bool begins = valid && (place == 0 || before != s - 1);
            // not the first token of its group here, and not the next one either
            const bool apart = begins && place > 0 && before >= 0 && before / group == s / group;
            int n = 0;
            if (begins && !apart) {
                n = 1;
                while (place + n < group && lane + n < known && slot[1 + lane + n] == s + n) ++n;
            }
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, n > 0);
            if (n > 0) run[__popc(who & ((1u << lane) - 1u))] = make_int2(lane, n);
            const int end = __reduce_max_sync(0xFFFFFFFFu, n ? lane + n : 0);
            if (lane == 0) runs = __popc(who), run_end = end;
            if ((s != -1 && !valid) || apart) raise_device_error(a.err, W4A16_DEVERR_SLOT);
        }
        __syncthreads();
    }
    const int heads = a.cache.heads, first_item = blockIdx.y * plan.items, items = min(plan.items, 2 * heads - first_item);
    if (first_item < heads) {
        if (turned) angles_of(a, t0, run_end, angles);
        __syncthreads();
    }

    // --- one run of one head at a time ------------------------------------------
    for (int i = warp; i < runs * items; i += kThreads / 32) {
        const int r = i / items, item = first_item + i - r * items;
        const bool key = item < heads;
        const int head = key ? item : item - heads;
        const int first = run[r].x, units = run[r].y * per_head;
        const int s = slot[1 + first];
        const int64_t block = s / a.cache.page;
        const int place = s - static_cast<int>(block) * a.cache.page;  // of the run's first token in its block
        const int of = plan.magic ? static_cast<int>(__umulhi(place, plan.magic)) : place, held = place - of * group;
        float* const scale_at = key ? a.cache.k_scale + block * a.cache.ks_block + of * a.cache.ks_group + head * a.cache.ks_head
                                    : a.cache.v_scale + block * a.cache.vs_block + of * a.cache.vs_group + head * a.cache.vs_head;
        const float old = held ? *scale_at : 0.f;
        const int64_t token_stride = key ? a.k_token : a.v_token;
        const uint16_t* const src = (key ? a.k + head * a.k_head : a.v + head * a.v_head) + (t0 + first) * token_stride;
        uint8_t* const dst = (key ? static_cast<uint8_t*>(a.cache.k) + block * a.cache.k_block + head * a.cache.k_head
                                  : static_cast<uint8_t*>(a.cache.v) + block * a.cache.v_block + head * a.cache.v_head);
        const int64_t code_stride = key ? a.cache.k_token : a.cache.v_token;
        const bool turns = key && turned;
        const auto unit = [&](int u, int& token) {
            token = static_cast<int>(u * plan.unit_magic >> 16);
            return place_of(u - token * per_head, a.dim, a.rotary, turns, a.interleaved);
        };
        const auto load = [&](int u, uint4& v0, uint4& v1) {
            int token;
            const Place at = unit(u, token);
            v0 = *reinterpret_cast<const uint4*>(src + token * token_stride + at.d0);
            v1 = *reinterpret_cast<const uint4*>(src + token * token_stride + at.d1);
        };
        uint4 v0[kKeep], v1[kKeep];
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
            v0[j] = v1[j] = make_uint4(0u, 0u, 0u, 0u);
            if (j * 32 + lane < units) load(j * 32 + lane, v0[j], v1[j]);
        }
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < kKeep; ++j) m = largest(largest(m, v0[j]), v1[j]);
        for (int u = kKeep * 32 + lane; u < units; u += 32) {
            uint4 x0, x1;
            load(u, x0, x1);
            m = largest(largest(m, x0), x1);
        }
        m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16)) << 16;
        int e = exponent_for<INT8>(m);
        if (turns && m < 0x7F800000u) {
            const float inv = exp2i(-e), most2 = INT8 ? 127.f * 127.f : 448.f * 448.f;
            bool over = false;
#pragma unroll
            for (int j = 0; j < kKeep; ++j) {
                int token;
                const Place at = unit(j * 32 + lane, token);
                over |= longer(v0[j], v1[j], at, a.rotary, inv, most2);
            }
            for (int u = kKeep * 32 + lane; u < units; u += 32) {
                uint4 x0, x1;
                int token;
                load(u, x0, x1);
                over |= longer(x0, x1, unit(u, token), a.rotary, inv, most2);
            }
            e += __any_sync(0xFFFFFFFFu, over) ? 1 : 0;
        }
        const uint32_t old_bits = __float_as_uint(old) & 0x7FFFFFFFu;
        if (old_bits) e = max(e, static_cast<int>(old_bits >> 23) - 127 + ((old_bits & 0x7FFFFFu) ? 1 : 0));
        // (a scale of 2^-126 or less so far is raised to that)
        const float S = m >= 0x7F800000u || e > 127 ? __uint_as_float(0x7FFFFFFFu) : exp2i(e);
        if (held && __float_as_uint(S) != __float_as_uint(old)) {
            const float ratio = old / S;
            for (int u = lane; u < held * per_head; u += 32) {
                const int token = static_cast<int>(u * plan.unit_magic >> 16);
                uint4* const at = reinterpret_cast<uint4*>(dst + (place - held + token) * code_stride + (u - token * per_head) * 16);
                *at = again<INT8>(*at, ratio);
            }
        }
        if (lane == 0) *scale_at = S;
        const float inv = 1.f / S;
        const auto store = [&](int u, const uint4& x0, const uint4& x1) {
            int token;
            const Place at = unit(u, token);
            float p[8], q[8];
            unpack8(x0, p);
            unpack8(x1, q);
            if (turns) turn(p, q, at, angles + (first + token) * 4 * turned, a.rotary);
            uint8_t* const to = dst + (place + token) * code_stride;
            *reinterpret_cast<uint2*>(to + at.d0) = codes_of<INT8>(p, inv);
            *reinterpret_cast<uint2*>(to + at.d1) = codes_of<INT8>(q, inv);
        };
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
            if (j * 32 + lane < units) store(j * 32 + lane, v0[j], v1[j]);
        for (int u = kKeep * 32 + lane; u < units; u += 32) {
            uint4 x0, x1;
            load(u, x0, x1);
            store(u, x0, x1);
        }
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_scaled_append(const ScaledAppendArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    const int per_head = a.dim / 16, half = a.rotary / 2;
    AppendPlan plan{};
    plan.unit_magic = (65536 + per_head - 1) / per_head;
    plan.magic = a.cache.heads ? group_magic(a.cache.group) : 0u;
    // a chunk for every SM at least, of at most kChunk tokens
    plan.chunk = kChunk;
    while (plan.chunk > 1 && (a.T + plan.chunk - 1) / plan.chunk < dev.sms) plan.chunk /= 2;
    const int64_t chunks = (a.T + plan.chunk - 1) / plan.chunk;
    // where those are few, the heads of a chunk over several CTAs
    int parts = 1;
    const int all = 2 * a.cache.heads, units = a.q_heads * per_head;
    while (parts * 8 < all && chunks * parts < dev.sms) parts *= 2;
    plan.items = (all + parts - 1) / parts;
    plan.kv_parts = all ? (all + plan.items - 1) / plan.items : 0;
    parts = (units + kThreads - 1) / kThreads;
    while (units && units / parts > 64 && chunks * parts < dev.sms) parts *= 2;
    plan.range = parts ? (units + parts - 1) / parts : 1;
    const int q_parts = units ? (units + plan.range - 1) / plan.range : 0;
    const int tokens = plan.chunk + (a.cache.heads ? a.cache.group - 1 : 0);
    const int smem = std::max(tokens * half * 8, 16);
    auto* kernel = a.cache.dtype == W4A16_CACHE_INT8 ? k_scaled_append<true> : k_scaled_append<false>;
    const cudaError_t rc = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (rc != cudaSuccess) return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(plan.kv_parts + q_parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, plan);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4a16
