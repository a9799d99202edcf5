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
//
// Measured on one GB300 (copies run at 6.77 TB/s), 32 query heads over 8 of 128 dims: 17002
// tokens of ragged prompts 71.9 us, 383 MB at 5.3 TB/s (0.79 of the copy rate); of them keys
// and values alone 37 us for 209 MB: every run is read, searched, and written by one warp, whose
// long reads have 24 warps an SM to hide behind (of 10 cycles between a
// warp's issues 3.2 wait for memory; the issue slots are half busy).  One token 4.2 us (3.8 in a graph): launch, slots and positions,
// then values, one after another.  Slower for the prompts: chunks of 16 tokens 74.9 us, four
// CTAs an SM, which spill 306 bytes, 83; CTAs that stay and bring the next chunk to L2 94 to
// 167; the next run's values in registers 73.  (Three spill 84 to 88 bytes.)
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
    int chunk, kv_parts, items;    // tokens of a CTA for keys and values; CTAs of a chunk, heads (key, then value) of each
    int q_chunk, q_parts, range;   // tokens of one for queries; CTAs of those, units of each
    unsigned kv_ctas;              // all for keys and values
    int turns;                     // CTAs of a chunk for keys, values and queries follow one another (chunks alike), else
};                                 // those for queries come last

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

// What the angles of a CTA's tokens are made of, in shared memory: a thread that read its
// positions one after another waited for each (4 us of a CTA's 12).
struct Angles {
    float freq[128];
    int axis[128];                             // of a pair
    int position[4][kChunk + kMostGroup];      // of a token, from the chunk's first on
};
__device__ __forceinline__ void request_angles(const ScaledAppendArgs& a, int64_t t0, int tokens, Angles& x) {
    const int half = a.rotary / 2;
    if (static_cast<int>(threadIdx.x) < half) {
        int axis = 0;
        while (axis < 3 && static_cast<int>(threadIdx.x) >= a.axis_end[axis]) ++axis;
        x.freq[threadIdx.x] = a.inv_freq[threadIdx.x];
        x.axis[threadIdx.x] = axis;
    }
    for (int i = threadIdx.x; i < tokens; i += kThreads)
#pragma unroll
        for (int axis = 0; axis < 4; ++axis)
            if (axis == 0 || a.axis_end[axis] > a.axis_end[axis - 1]) x.position[axis][i] = a.positions[axis * a.axis_stride + t0 + i];
}
// cos and sin of pos * f as turn_of() forms them, and what the last rounding of the half
// turns takes away put back by its first order: a code is rounded once from a key that is
// as good as 32 bits allow, so fewer of them lie on the other side of a tie.
__device__ __forceinline__ float2 exact_turn_of(int pos, float f) {
    float high, low;
    if (static_cast<unsigned>(pos) < (1u << 24)) {
        const float gh = f * kInvPiHi;
        const float gl = fmaf(f, kInvPiLo, fmaf(f, kInvPiHi, -gh));
        const float p = static_cast<float>(pos);  // exact
        const float th = p * gh;
        const float x = th - 2.f * rintf(0.5f * th), y = fmaf(p, gl, fmaf(p, gh, -th));  // x is exact
        high = x + y;
        const float z = high - x;
        low = (x - (high - z)) + (y - z);
    } else {
        const double t = static_cast<double>(pos) * (static_cast<double>(f) * 0.31830988618379067154), r = t - 2.0 * rint(0.5 * t);
        high = static_cast<float>(r);
        low = static_cast<float>(r - static_cast<double>(high));
    }
    float2 cs;
    sincospif(high, &cs.y, &cs.x);
    const float d = 3.14159274f * low;
    return make_float2(fmaf(-cs.y, d, cs.x), fmaf(cs.x, d, cs.y));
}
// The angles of tokens from .. to - 1 of the chunk: the i-th float4 (cos, sin, cos, sin) of all
// units of a token next to one another.
__device__ __forceinline__ void angles_of(const ScaledAppendArgs& a, const Angles& x, int from, int to, float4* angles) {
    const int half = a.rotary / 2, turned = a.rotary / 16;
    for (int i = from * half + threadIdx.x; i < to * half; i += kThreads) {
        const int token = i / half, pair = i - token * half;
        const float2 c = exact_turn_of(x.position[x.axis[pair]][token], x.freq[pair]);
        float4* cs = angles + token * 4 * turned;
        cs += a.interleaved ? (pair & 3) / 2 * 2 * turned + pair / 4 : (pair & 7) / 2 * turned + pair / 8;
        reinterpret_cast<float2*>(cs)[pair & 1] = c;
    }
}

// the larger magnitudes of bf16 pairs (of a NaN: a NaN)
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("{.reg .b32 x, y;\n abs.bf16x2 x, %1;\n abs.bf16x2 y, %2;\n max.NaN.bf16x2 %0, x, y;}" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t largest(uint32_t m, const uint4& v) { return larger(m, larger(larger(v.x, v.y), larger(v.z, v.w))); }

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

__device__ __forceinline__ void scale8(float (&x)[8], float f) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        asm("{.reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;}"
            : "+f"(x[i]), "+f"(x[i + 1])
            : "f"(f));
}
template <bool INT8>
__device__ __forceinline__ uint2 codes_of(const float (&x)[8]) {
    return make_uint2(f32_to_codes<INT8>(x[0], x[1], x[2], x[3]), f32_to_codes<INT8>(x[4], x[5], x[6], x[7]));
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

// New tokens of one group.
struct Run {
    int first, tokens;         // of the chunk
    int held;                  // places of the group before the first
    int64_t k, v, ks, vs;      // where the first one's codes and scales begin (of head 0)
};

// PER_SM: CTAs of an SM.  Three where there are many tokens (17002: 72.1 us against 74.7 with
// two), two where a single CTA's time counts, whose registers then hold all that it needs (one
// token 3.7 against 4.3).
template <bool INT8, int PER_SM>
__global__ void __launch_bounds__(kThreads, PER_SM) k_scaled_append(const ScaledAppendArgs a, const AppendPlan plan) {
    extern __shared__ __align__(16) float4 angles[];
    __shared__ int slot[kChunk + kMostGroup + 1];  // of the token before the chunk, then from its first on
    __shared__ Run run[kChunk];
    __shared__ int runs, run_end;
    __shared__ Angles terms;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_head = a.dim / 16, turned = a.rotary / 16;
    // Where there are many, CTAs of keys and of queries take turns, so that the ones copy while the
    // others look for their scales.
    bool queries;
    int part;
    int64_t t0;
    if (plan.turns) {
        const unsigned parts = plan.kv_parts + plan.q_parts;
        t0 = static_cast<int64_t>(blockIdx.x / parts) * plan.chunk;
        part = blockIdx.x % parts;
        queries = part >= plan.kv_parts;
        if (queries) part -= plan.kv_parts;
    } else {
        queries = blockIdx.x >= plan.kv_ctas;
        const unsigned id = queries ? blockIdx.x - plan.kv_ctas : blockIdx.x, parts = queries ? plan.q_parts : plan.kv_parts;
        t0 = static_cast<int64_t>(id / parts) * (queries ? plan.q_chunk : plan.chunk);
        part = id % parts;
    }
    const int chunk = queries ? plan.q_chunk : plan.chunk;
    const int64_t left = a.T - t0;
    const int here = left < chunk ? static_cast<int>(left) : chunk;
    grid_dependency_wait();
    grid_dependents_launch();

    if (queries) {
        // --- queries -----------------------------------------------------------
        const int u0 = part * plan.range, range = min(plan.range, a.q_heads * per_head - u0);
        const int step = kThreads / range, mine = static_cast<int>(threadIdx.x) / range;
        const int u = u0 + static_cast<int>(threadIdx.x) - mine * range, head = u / per_head;
        const Place at = place_of(u - head * per_head, a.dim, a.rotary, turned > 0, a.interleaved);
        const bool idle = mine >= step;
        const uint16_t* src = a.q + (t0 + mine) * a.q_token + head * a.q_head;
        uint16_t* dst = a.q_out + (t0 + mine) * a.qo_token + head * a.qo_head;
        const int64_t src_step = step * a.q_token, dst_step = step * a.qo_token;
        const float4* cs = angles + mine * 4 * turned;
        constexpr int kBatch = 4;
        // the next tokens requested before these are written
        const auto load = [&](uint4 (&v0)[kBatch], uint4 (&v1)[kBatch], int from) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (idle || from + j * step >= here) continue;
                v0[j] = *reinterpret_cast<const uint4*>(src + at.d0);
                v1[j] = *reinterpret_cast<const uint4*>(src + at.d1);
                src += src_step;
            }
        };
        const auto store = [&](const uint4 (&v0)[kBatch], const uint4 (&v1)[kBatch], int from) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (idle || from + j * step >= here) continue;
                float p[8], q[8];
                unpack8(v0[j], p);
                unpack8(v1[j], q);
                turn(p, q, at, cs, a.rotary);
                *reinterpret_cast<uint4*>(dst + at.d0) = pack8(p);
                *reinterpret_cast<uint4*>(dst + at.d1) = pack8(q);
                dst += dst_step, cs += step * 4 * turned;
            }
        };
        uint4 v0[kBatch], v1[kBatch];
        load(v0, v1, mine);
        if (turned) {
            request_angles(a, t0, here, terms);
            __syncthreads();
            angles_of(a, terms, 0, here, angles);
            __syncthreads();
        }
        for (int from = mine; from < here; from += kBatch * step) {
            if (from != mine) load(v0, v1, from);
            store(v0, v1, from);
        }
        return;
    }

    // --- the runs that begin in the chunk ---------------------------------------
    const int group = a.cache.group;
    const int heads = a.cache.heads, first_item = part * plan.items, items = min(plan.items, 2 * heads - first_item);
    const bool turns_any = first_item < heads && turned;
    {
        const int most = chunk + group - 1, known = left < most ? static_cast<int>(left) : most;
        for (int i = threadIdx.x; i <= known; i += kThreads) slot[i] = i || t0 ? a.slots[t0 + i - 1] : -1;
        if (turns_any) request_angles(a, t0, known, terms);
        __syncthreads();
        if (warp == 0) {
            const int s = lane < here ? slot[1 + lane] : -1, before = lane < here ? slot[lane] : -1;
            const bool valid = s >= 0 && s < a.cache.blocks * a.cache.page;
            const int place = valid ? s % group : 0;
            const bool begins = valid && (place == 0 || before != s - 1);
            // in the group of the token before it, whose warp has that group, but not behind it: not
            // stored, nor what goes on from it (which begins nothing)
            const bool apart = begins && before >= 0 && before / group == s / group;
            int n = 0;
            if (begins && !apart) {
                n = 1;
                while (place + n < group && lane + n < known && slot[1 + lane + n] == s + n) ++n;
            }
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, n > 0);
            if (n > 0) {
                const w4a16_scaled_cache& c = a.cache;
                const int64_t block = s / c.page;
                const int in = s - static_cast<int>(block) * c.page;
                const int64_t of = in / group;
                run[__popc(who & ((1u << lane) - 1u))] = Run{lane, n, place, block * c.k_block + in * c.k_token, block * c.v_block + in * c.v_token,
                                                             block * c.ks_block + of * c.ks_group, block * c.vs_block + of * c.vs_group};
            }
            const int end = __reduce_max_sync(0xFFFFFFFFu, n ? lane + n : 0);
            if (lane == 0) runs = __popc(who), run_end = end;
            if ((s != -1 && !valid) || apart) raise_device_error(a.err, W4A16_DEVERR_SLOT);
        }
        __syncthreads();
    }
    // --- one run of one head at a time ------------------------------------------
    // A step takes as many tokens as have lanes for all units of a head; this lane's unit:
    const int tps = 32 / per_head, mine = lane / per_head, unit = lane - mine * per_head;
    const Place turning = place_of(unit, a.dim, a.rotary, turned > 0, a.interleaved), still = place_of(unit, a.dim, a.rotary, false, a.interleaved);
    struct Item {
        const uint16_t* src;  // this lane's first token
        int64_t step;         // to that of the next step
        int run, head, left;  // left: tokens from this lane's first on (at most 0: none)
        bool key;
    };
    const auto open = [&](int i) {
        Item x;
        x.run = i / items;
        const int item = first_item + i - x.run * items;
        x.key = item < heads;
        x.head = x.key ? item : item - heads;
        const int64_t stride = x.key ? a.k_token : a.v_token;
        x.src = (x.key ? a.k + x.head * a.k_head : a.v + x.head * a.v_head) + (t0 + run[x.run].first + mine) * stride;
        x.step = tps * stride;
        x.left = mine < tps ? run[x.run].tokens - mine : 0;
        return x;
    };
    const auto fetch = [&](const Item& x, uint4 (&v0)[kKeep], uint4 (&v1)[kKeep]) {
        const Place at = x.key ? turning : still;
        const uint16_t* src = x.src;
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
            v0[j] = v1[j] = make_uint4(0u, 0u, 0u, 0u);
            if (j * tps < x.left) {
                v0[j] = *reinterpret_cast<const uint4*>(src + at.d0);
                v1[j] = *reinterpret_cast<const uint4*>(src + at.d1);
                src += x.step;
            }
        }
    };
    const auto work = [&](const Item& x, const uint4 (&v0)[kKeep], const uint4 (&v1)[kKeep]) {
        const bool turns = x.key && turned;
        const Place at = x.key ? turning : still;
        const Run& r = run[x.run];
        const int held = r.held;
        float* const scale_at = x.key ? a.cache.k_scale + r.ks + x.head * a.cache.ks_head : a.cache.v_scale + r.vs + x.head * a.cache.vs_head;
        const float old = held ? *scale_at : 0.f;
        // steps past kKeep: their values are read again each time
        const auto rest = [&](auto&& take) {
            if (kKeep * tps >= r.tokens) return;
            const uint16_t* src = x.src + kKeep * x.step;
            for (int j = kKeep; j * tps < x.left; ++j, src += x.step)
                take(j, *reinterpret_cast<const uint4*>(src + at.d0), *reinterpret_cast<const uint4*>(src + at.d1));
            __syncwarp();
        };
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < kKeep; ++j) m = largest(largest(m, v0[j]), v1[j]);
        rest([&](int, const uint4& x0, const uint4& x1) { m = largest(largest(m, x0), x1); });
        m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16)) << 16;
        int e = exponent_for<INT8>(m);
        constexpr float kMost = INT8 ? 127.f : 448.f;
        // (no pair is longer than sqrt(2) times its larger value)
        if (turns && m < 0x7F800000u && __uint_as_float(m) * exp2i(-e) > 0.7f * kMost) {
            const float inv = exp2i(-e);
            bool over = false;
#pragma unroll
            for (int j = 0; j < kKeep; ++j) over |= longer(v0[j], v1[j], at, a.rotary, inv, kMost * kMost);
            rest([&](int, const uint4& x0, const uint4& x1) { over |= longer(x0, x1, at, a.rotary, inv, kMost * kMost); });
            e += __any_sync(0xFFFFFFFFu, over) ? 1 : 0;
        }
        const uint32_t old_bits = __float_as_uint(old) & 0x7FFFFFFFu;
        if (old_bits) e = max(e, static_cast<int>(old_bits >> 23) - 127 + ((old_bits & 0x7FFFFFu) ? 1 : 0));
        // (a scale of 2^-126 or less so far is raised to that)
        const float S = m >= 0x7F800000u || e > 127 ? __uint_as_float(0x7FFFFFFFu) : exp2i(e);
        uint8_t* dst = (x.key ? static_cast<uint8_t*>(a.cache.k) + r.k + x.head * a.cache.k_head : static_cast<uint8_t*>(a.cache.v) + r.v + x.head * a.cache.v_head);
        const int64_t code_stride = x.key ? a.cache.k_token : a.cache.v_token;
        if (held && __float_as_uint(S) != __float_as_uint(old)) {
            const float ratio = old / S;
            for (int before = held - mine; before > 0 && mine < tps; before -= tps) {
                uint4* const codes = reinterpret_cast<uint4*>(dst - before * code_stride + unit * 16);
                *codes = again<INT8>(*codes, ratio);
            }
        }
        if (lane == 0) *scale_at = S;
        // 1 / S (2^-127 is no normal number)
        const float inv = isnan(S) ? S : e == 127 ? __uint_as_float(0x00400000u) : exp2i(-e);
        dst += mine * code_stride;
        const int64_t dst_step = tps * code_stride;
        const float4* cs = angles + (r.first + mine) * 4 * turned;
        const auto put = [&](const uint4& x0, const uint4& x1) {
            float p[8], q[8];
            unpack8(x0, p);
            unpack8(x1, q);
            scale8(p, inv), scale8(q, inv);  // first: a pair of large values turns past what a float holds
            if (turns) turn(p, q, at, cs, a.rotary);
            *reinterpret_cast<uint2*>(dst + at.d0) = codes_of<INT8>(p);
            *reinterpret_cast<uint2*>(dst + at.d1) = codes_of<INT8>(q);
            dst += dst_step, cs += tps * 4 * turned;
        };
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
            if (j * tps < x.left) put(v0[j], v1[j]);
        rest([&](int, const uint4& x0, const uint4& x1) { put(x0, x1); });
        __syncwarp();
    };
    const int all = runs * items;
    uint4 v0[kKeep], v1[kKeep];
    Item now{};
    if (warp < all) now = open(warp), fetch(now, v0, v1);
    if (turns_any) {
        angles_of(a, terms, 0, run_end, angles);
        __syncthreads();
    }
    for (int i = warp; i < all; i += kThreads / 32) {
        if (i != warp) now = open(i), fetch(now, v0, v1);
        work(now, v0, v1);
    }
}

}  // namespace

cudaError_t launch_scaled_append(const ScaledAppendArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    const int per_head = a.dim / 16, half = a.rotary / 2;
    AppendPlan plan{};
    // Keys and values apart (the ones wait for angles), a head for every warp at least.  Chunks of
    // one token, of as many as leave no more CTAs than run at once, kChunk at most.
    const int all = 2 * a.cache.heads, units = a.q_heads * per_head;
    const auto chunks = [&](int chunk) { return (a.T + chunk - 1) / chunk; };
    plan.kv_parts = std::max(2, (all + kThreads / 32 - 1) / (kThreads / 32));
    plan.items = (all + plan.kv_parts - 1) / plan.kv_parts;
    plan.kv_parts = (all + plan.items - 1) / plan.items;
    plan.chunk = 1;
    while (plan.chunk < kChunk && chunks(plan.chunk) * plan.kv_parts > 2 * dev.sms) plan.chunk *= 2;
    while (plan.kv_parts > 2 && chunks(plan.chunk) * plan.kv_parts > 2 * dev.sms) {
        plan.items *= 2;
        plan.kv_parts = (all + plan.items - 1) / plan.items;
    }
    plan.q_parts = std::max(1, (units + kThreads - 1) / kThreads);
    plan.q_chunk = 1;
    const int64_t room = std::max<int64_t>(2 * dev.sms - chunks(plan.chunk) * plan.kv_parts, dev.sms / 4);  // beside those
    while (plan.q_chunk < kChunk && chunks(plan.q_chunk) * plan.q_parts > room) plan.q_chunk *= 2;
    while (units / plan.q_parts > 64 && chunks(plan.q_chunk) * plan.q_parts * 2 <= room) plan.q_parts *= 2;
    plan.range = std::max(1, (units + plan.q_parts - 1) / plan.q_parts);
    plan.q_parts = (units + plan.range - 1) / plan.range;
    plan.turns = plan.chunk == kChunk && plan.q_chunk == kChunk;
    plan.kv_ctas = static_cast<unsigned>(chunks(plan.chunk) * plan.kv_parts);
    const int64_t ctas = plan.kv_ctas + chunks(plan.q_chunk) * plan.q_parts;
    if (ctas >= int64_t(1) << 31) return cudaErrorInvalidConfiguration;  // (2^31 tokens of 65536 heads, all one by strides of 0)
    const bool many = ctas > 2 * dev.sms;
    const int tokens = std::max(plan.chunk + a.cache.group - 1, plan.q_chunk);
    const int smem = std::max(tokens * half * 8, 16);
    const bool int8 = a.cache.dtype == W4A16_CACHE_INT8;
    auto* kernel = many ? (int8 ? k_scaled_append<true, 3> : k_scaled_append<false, 3>) : int8 ? k_scaled_append<true, 2> : k_scaled_append<false, 2>;
    const cudaError_t rc = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (rc != cudaSuccess) return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
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
