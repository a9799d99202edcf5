// Attention of one new token per request over a paged key/value cache
// (w4a16_paged_attention): the kernels, for one cache type per translation unit.
//
// A row is one request, one key/value head and up to 8 * NT of the query
// heads that share it.  For the tokens j a row sees,
//     s_j = c q . k_j (log2 units),  m = max s_j,  p_j = 2^(s_j - m),
//     l = sum p_j,  o = sum p_j v_j,  out = o / l,
// in one pass: a larger m scales the running l and o by 2^(m_old - m).
// Parts (m, l, o) of disjoint token sets join the same way, in any grouping.
//
// Bound by HBM: each key and value is read once, for 2 * heads operations a
// byte at most.  So the kernels are built around the copies, tiles of 16
// tokens through a ring of cp.async stages that each warp has for itself:
//   - k_attention_shares: the tiles of all rows, one row after another, in
//     equal consecutive shares for the warps of the whole GPU, whatever the
//     lengths are.  A row inside a share its warp finishes alone; of the rows
//     at the ends of a share it leaves parts in the workspace.  The ring runs
//     on across rows, and no warp waits for another.
//   - k_attention_join: a second launch joins those parts, always in the
//     order of the tokens.
//   - k_attention_rows: where no row can have many tiles, one to eight warps of
//     a CTA for each row, or, where rows are few, a cluster of up to eight such
//     CTAs, joined through shared memory: no shares, no second launch.
// The products run on the warp MMA with the keys as the 16-row operand
// (tokens) and the heads as its 8 columns: one product covers 8 query heads,
// and the transposed second product (values^T times p^T) takes the
// probabilities from the accumulators by one 8x8 transpose in registers.
// (tcgen05 would want 64 or more query rows; here there are 1 to 16.)
//
// Measured on one GB300 (copies run at 6.67 TB/s) in a CUDA graph, 32 query
// heads over 8 of 128 dims: one request of 131072 tokens in bf16 92 us (5.85
// TB/s), 128 requests of 0 to 8192 tokens over e4m3 125 us (5.82 TB/s; 58 % of
// the issue slots, 18 % of the tensor pipe), 16 requests of 0 to 4096 tokens
// 26 us (15 us of it at the rate of HBM, the rest the two launches), one request
// of 300 tokens 4.9 us.
// Registers: all instances but those of 16 heads of 256 dims (24 bytes spilled
// by the shares over bf16, 104 over e4m3) and 16 of 192 over e4m3 (32) hold what
// they need.
#pragma once

#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "paged_attention.h"

namespace w4a16 {
namespace {

constexpr int kMinCost = 3;     // a warp's share at least
constexpr int kRowTiles = 8;    // rows kernel: tiles of a warp at most
constexpr int kRowEnough = 2;   // and where one CTA is enough

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&d)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(addr)
                 : "memory");
}
// 8x8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(m - top) of a part that is not empty (m may be infinite)
__device__ __forceinline__ float part_factor(float m, float top) { return m == top ? 1.f : exp2_fast(m - top); }
// two e4m3 codes (low and high byte) as an fp16 pair, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(v)));
    return d;
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
template <bool E4M3>
__device__ __forceinline__ void attn_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (E4M3) {
        mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
    } else {
        const uint32_t a[4] = {a0, a1, a2, a3};
        mma_bf16_16816(d, a, b0, b1, d);
    }
}

// byte offset of chunk c of row r in a tile whose rows have CH chunks: eight
// rows reading one chunk hit eight different 16-byte bank groups
template <int CH>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
    const int f = (CH % 8 == 0) ? (r & 7) : ((r >> 1) & 3);
    return static_cast<uint32_t>((r * CH + (c ^ f)) * 16);
}

template <bool E4M3, int DP, int NT>
struct AttnShape {
    static constexpr int kHeads = 8 * NT;
    static constexpr int kSteps = DP / 16;                     // 16-dim steps of a head
    // 16-byte chunks of a row in shared memory (six would not swizzle: eight)
    static constexpr int kChunks = E4M3 && DP == 96 ? 8 : DP * (E4M3 ? 1 : 2) / 16;
    static constexpr int kRowBytes = kChunks * 16;
    static constexpr int kStageBytes = 2 * kTile * kRowBytes;  // keys, then values
    static constexpr int kPartFloats = kHeads * (DP + 2);
    // shares: one CTA an SM, of as many warps as its registers allow (the accumulators'
    // size decides) with rings of three stages or more
    static constexpr int kShareWarps = 4 * (E4M3 ? (NT == 1 ? (DP == 64 ? 4 : DP <= 128 ? 3 : 2) : (DP == 64 ? 3 : 2))
                                                 : (DP == 64 ? 3 : DP <= 128 ? 2 : 1));
    static constexpr int kFit = 226 * 1024 / (kShareWarps * kStageBytes);
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kSmem = kShareWarps * kStages * kStageBytes;
    // rows: one CTA an SM
    static constexpr int kRowWarps = kStageBytes > 12288 ? 4 : 8;
    static constexpr int kRowFit = 225 * 1024 / (kRowWarps * kStageBytes);
    static constexpr int kRowStages = kRowFit > 4 ? 4 : kRowFit;
    static constexpr int kRowRing = kRowStages * kStageBytes;  // of a warp
    static constexpr int kRowSmem = kRowWarps * kRowRing;
    static constexpr int kPartBytes = kHeads * DP * 4;
    static constexpr bool kClusters = kRowRing >= 2 * kPartBytes;  // room for the CTA's part behind a warp's
    static_assert(kStages >= 3, "ring too short");
    static_assert(kRowStages >= 2 && kRowRing >= kPartBytes, "no room for a warp's part");
    static_assert(160 * kShareWarps <= most_workers(DP), "workspace");
};

// What one request looks like: its visible tokens [start, len), in tiles from
// tile0 on.
struct Request {
    int len, start, tile0, tiles;
};

__device__ __forceinline__ Request request_of(const AttentionArgs& a, int b, bool& bad) {
    Request q;
    const int len = a.kv_len[b];
    bad |= len < 0 || len > a.most;
    q.len = min(max(len, 0), a.most);
    q.start = a.window > 0 ? max(q.len - a.window, 0) : 0;
    q.tile0 = q.start / kTile;
    q.tiles = q.len > 0 ? (q.len - 1) / kTile + 1 - q.tile0 : 0;
    return q;
}

// Which heads row `row` of a request stands for.
struct Heads {
    int hk, first, n;  // key/value head, first query head, how many
};
template <int HEADS>
__device__ __forceinline__ Heads heads_of(const AttentionArgs& a, int row) {
    const int G = a.q_heads / a.cache.heads, chunks = (G + HEADS - 1) / HEADS;
    Heads h;
    h.hk = row / chunks;
    const int chunk = row - h.hk * chunks;
    h.first = h.hk * G + chunk * HEADS;
    h.n = min(HEADS, G - chunk * HEADS);
    return h;
}

__device__ __forceinline__ void store_empty(const AttentionArgs& a, int b, int head, int heads, int thread, int threads) {
    const int per = a.cache.dim / 8;
    for (int i = thread; i < heads * per; i += threads) {
        const int h = head + i / per, d = (i % per) * 8;
        *reinterpret_cast<uint4*>(a.out + b * a.out_request + h * a.out_head + d) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (a.lse)
        for (int h = thread; h < heads; h += threads) a.lse[static_cast<int64_t>(b) * a.q_heads + head + h] = -INFINITY;
}

// 16 dims of 8 heads from the accumulators (row r and r + 8 by columns 2c,
// 2c + 1) times the heads' factors, transposed to dims along the lanes of a
// head and stored; `out`: the row of head r's output, null for none.
template <bool E4M3>
__device__ __forceinline__ void store_dims(const float4& o, float f0, float f1, uint16_t* out, int c) {
    const __nv_bfloat162 p0 = __floats2bfloat162_rn(o.x * f0, o.y * f1), p1 = __floats2bfloat162_rn(o.z * f0, o.w * f1);
    const uint32_t v0 = transpose_8x8(*reinterpret_cast<const uint32_t*>(&p0));
    const uint32_t v1 = transpose_8x8(*reinterpret_cast<const uint32_t*>(&p1));
    if (!out) return;
    if (E4M3) {  // rows of the product: even dims, then odd ones
        *reinterpret_cast<uint2*>(out + 4 * c) = make_uint2(__byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632));
    } else {
        *reinterpret_cast<uint32_t*>(out + 2 * c) = v0;
        *reinterpret_cast<uint32_t*>(out + 8 + 2 * c) = v1;
    }
}
template <bool E4M3>
__device__ __forceinline__ float lse_of(float m, float l) {
    return l != 0.f ? (m + (log2f(l) - (E4M3 ? kE4m3Bias : 0.f))) * 0.6931471805599453f : -INFINITY;
}

// The arithmetic of a warp on tiles of one row.  Lane 4 r + c.
template <bool E4M3, int DP, int NT>
struct RowMath {
    using Sh = AttnShape<E4M3, DP, NT>;
    static constexpr int CH = Sh::kChunks, KS = Sh::kSteps;
    uint32_t qf[NT][KS][2];              // queries as B fragments (columns: heads)
    float sl[NT][2];                     // score scale of columns 2c, 2c + 1
    float m[NT][2], l[NT][2];            // of columns 2c, 2c + 1 (l: of this lane's tokens until reduced)
    float4 o[NT][KS];                    // dims r, r + 8 (e4m3: 2r, 2r + 1) by columns 2c, 2c + 1

    // requests the queries and clears the sums
    __device__ __forceinline__ void begin(const AttentionArgs& a, int b, const Heads& hd, int lane) {
        const int r = lane >> 2, c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint16_t* qp = a.q + b * a.q_request + (hd.first + n * 8 + r) * a.q_head;
            const bool have = n * 8 + r < hd.n;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[n][k][0] = qf[n][k][1] = 0u;
                if (have && k * 16 < a.cache.dim) {
                    // bf16: dims 2c, 2c + 1 and 8 further; e4m3: the four dims whose codes one word holds
                    const int d = k * 16 + (E4M3 ? 4 * c : 2 * c);
                    qf[n][k][0] = *reinterpret_cast<const uint32_t*>(qp + d);
                    qf[n][k][1] = *reinterpret_cast<const uint32_t*>(qp + d + (E4M3 ? 2 : 8));
                }
                o[n][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
            }
        }
    }

    // makes the queries that begin() requested into operands
    __device__ __forceinline__ void ready(const AttentionArgs& a, int hk, int lane) {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            sl[n][0] = sl[n][1] = a.scale * 1.4426950408889634f * (E4M3 ? a.cache.k_scale[hk] : 1.f);
            if (E4M3) {
                // to fp16, scaled by a power of two that takes the head's largest into [2^14, 2^15)
                uint32_t big = 0u;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    big = __vmaxu2(big, __vmaxu2(qf[n][k][0] & 0x7FFF7FFFu, qf[n][k][1] & 0x7FFF7FFFu));
                big = max(big & 0xFFFFu, big >> 16);
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                const int sh = min(141 - min(static_cast<int>(big >> 7), 254), 126);
                const float up = exp2i(sh), down = exp2i(-sh);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t v = qf[n][k][e];
                        const __half2 h = __floats2half2_rn(bf16_to_f32(v & 0xFFFFu) * up, bf16_to_f32(v >> 16) * up);
                        qf[n][k][e] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                sl[n][0] *= __shfl_sync(0xFFFFFFFFu, down, 8 * c);
                sl[n][1] *= __shfl_sync(0xFFFFFFFFu, down, 8 * c + 4);
            }
        }
    }

    // the tile at kt (shared address): keys, then values; mask: tokens that count
    __device__ __forceinline__ void tile(uint32_t kt, uint32_t mask, int lane) {
        const uint32_t vt = kt + kTile * Sh::kRowBytes;
        const int r = lane >> 2;
        // two chains of products, where registers allow: the latency of one is a good part of a tile's
        constexpr bool kTwo = NT * KS <= 16;
        float s[NT][4], s1[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = s1[n][e] = 0.f;
        if (!E4M3) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t f[4];
                ldmatrix_x4(f, kt + tile_offset<CH>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
                for (int n = 0; n < NT; ++n) attn_mma<E4M3>(kTwo && (k & 1) ? s1[n] : s[n], f[0], f[1], f[2], f[3], qf[n][k][0], qf[n][k][1]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                uint32_t f[4];  // two chunks of 16 codes: rows r and r + 8 of each
                ldmatrix_x4(f, kt + tile_offset<CH>(lane & 15, k + (lane >> 4)));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t a0 = e4m3x2_to_f16x2(f[2 * j]), a2 = e4m3x2_to_f16x2(f[2 * j] >> 16);
                    const uint32_t a1 = e4m3x2_to_f16x2(f[2 * j + 1]), a3 = e4m3x2_to_f16x2(f[2 * j + 1] >> 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        attn_mma<E4M3>(kTwo && j ? s1[n] : s[n], a0, a1, a2, a3, qf[n][k + j][0], qf[n][k + j][1]);
                }
            }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = (s[n][e] + s1[n][e]) * sl[n][e & 1];
            if (mask != 0xFFFFu) {
                if (!((mask >> r) & 1u)) s[n][0] = s[n][1] = -INFINITY;
                if (!((mask >> (r + 8)) & 1u)) s[n][2] = s[n][3] = -INFINITY;
            }
            float top[2] = {fmaxf(s[n][0], s[n][2]), fmaxf(s[n][1], s[n][3])};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 4));
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 8));
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 16));
                top[e] = fmaxf(top[e], m[n][e]);
            }
            if (__any_sync(0xFFFFFFFFu, top[0] > m[n][0] || top[1] > m[n][1])) {
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    keep[e] = part_factor(m[n][e], top[e]);  // from -infinity: 0
                    m[n][e] = top[e];
                    l[n][e] *= keep[e];
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    o[n][k].x *= keep[0], o[n][k].y *= keep[1];
                    o[n][k].z *= keep[0], o[n][k].w *= keep[1];
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // the bias after the difference: m - 15 is not a float where m passes 2^24, and
                // the largest p would then be 2^16, which no fp16 holds
                s[n][e] -= m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1];
                s[n][e] = exp2_fast(E4M3 ? s[n][e] + kE4m3Bias : s[n][e]);
                l[n][e & 1] += s[n][e];
            }
            // to 16 bits for the second product, whose operands are of one type: that of the
            // values.  fp16 rounds p by 2^-11 of it, bf16 by 2^-8, about as much as the result's
            // own rounding; l takes the unrounded ones.  (131072 tokens in bf16: 0.0020 off in
            // all, 0.0017 with fp32 weights; over e4m3 no difference shows.)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t v;
                if (E4M3) {
                    const __half2 h = __floats2half2_rn(s[n][2 * e], s[n][2 * e + 1]);
                    v = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(s[n][2 * e], s[n][2 * e + 1]);
                    v = *reinterpret_cast<const uint32_t*>(&h);
                }
                pf[n][e] = transpose_8x8(v);
            }
        }
        auto add = [&](int n, int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            float d[4] = {o[n][k].x, o[n][k].y, o[n][k].z, o[n][k].w};
            attn_mma<E4M3>(d, a0, a1, a2, a3, pf[n][0], pf[n][1]);
            o[n][k] = make_float4(d[0], d[1], d[2], d[3]);
        };
        if (!E4M3) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t f[4];
                ldmatrix_x4_trans(f, vt + tile_offset<CH>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                for (int n = 0; n < NT; ++n) add(n, k, f[0], f[1], f[2], f[3]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                uint32_t f[4];  // chunk k: tokens 0..7, 8..15, then chunk k + 1
                ldmatrix_x4_trans(f, vt + tile_offset<CH>(lane & 15, k + (lane >> 4)));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // word: dims 2r, 2r + 1 of token 2c, then of token 2c + 1
                    const uint32_t x0 = e4m3x2_to_f16x2(f[2 * j]), x1 = e4m3x2_to_f16x2(f[2 * j] >> 16);
                    const uint32_t y0 = e4m3x2_to_f16x2(f[2 * j + 1]), y1 = e4m3x2_to_f16x2(f[2 * j + 1] >> 16);
                    const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
                    const uint32_t a2 = __byte_perm(y0, y1, 0x5410), a3 = __byte_perm(y0, y1, 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) add(n, k + j, a0, a1, a2, a3);
                }
            }
        }
    }

    __device__ __forceinline__ void reduce() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 16);
            }
    }

    // the row's result, all of its tokens seen (after reduce())
    __device__ __forceinline__ void finish(const AttentionArgs& a, int b, const Heads& hd, int lane) {
        const int r = lane >> 2, c = lane & 3;
        const float vs = E4M3 ? a.cache.v_scale[hd.hk] : 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[e] = l[n][e] != 0.f ? vs / l[n][e] : 0.f;
                const int h = n * 8 + 2 * c + e;
                if (a.lse && r == 0 && h < hd.n)
                    a.lse[static_cast<int64_t>(b) * a.q_heads + hd.first + h] = lse_of<E4M3>(m[n][e], l[n][e]);
            }
            uint16_t* out = a.out + b * a.out_request + (hd.first + n * 8 + r) * a.out_head;
            const bool have = n * 8 + r < hd.n;
#pragma unroll
            for (int k = 0; k < KS; ++k)
                store_dims<E4M3>(o[n][k], f[0], f[1], have && k * 16 < a.cache.dim ? out + k * 16 : nullptr, c);
        }
    }

    // the row's part (after reduce()): o, then m and l of every head
    __device__ __forceinline__ void store_part(float* part, float* pm, float* pl, int lane) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < KS; ++k) reinterpret_cast<float4*>(part)[(n * KS + k) * 32 + lane] = o[n][k];
            if (lane < 4) {
                reinterpret_cast<float2*>(pm)[n * 4 + lane] = make_float2(m[n][0], m[n][1]);
                reinterpret_cast<float2*>(pl)[n * 4 + lane] = make_float2(l[n][0], l[n][1]);
            }
        }
    }
};

// The block ids and the copies of consecutive tiles of a row.  Ids are loaded
// early: where a tile lies in one block, those of 32 tiles at once (lane i:
// tile base + i * step), else those of one tile's tokens (lanes i and i + 16:
// token i).
template <bool E4M3, int DP, int NT>
struct TileCopy {
    using Sh = AttnShape<E4M3, DP, NT>;
    static constexpr int CH = Sh::kChunks, kBytes = E4M3 ? 1 : 2;
    int base, id, place;

    static __device__ __forceinline__ bool aligned(const AttentionArgs& a) { return a.cache.page % kTile == 0; }

    // the ids for tile t (tiles of the row step apart, below t1)
    __device__ __forceinline__ void look_up(const AttentionArgs& a, int b, const Request& q, int t, int t1, int step, int lane) {
        base = t;
        const bool whole = aligned(a);
        const int tile = whole ? t + lane * step : t;
        const int token = (q.tile0 + tile) * kTile + (whole ? 0 : lane & 15);
        const int col = static_cast<int>(static_cast<unsigned>(token) / static_cast<unsigned>(a.cache.page));
        place = token - col * a.cache.page;
        id = -1;
        if (whole ? tile < t1 : token >= q.start && token < q.len) {
            id = a.block_table[b * a.table_stride + col];
            if (id < 0) id = -2;
        }
    }
    // whether look_up has to come before copy(t)
    __device__ __forceinline__ bool wants(const AttentionArgs& a, int t, int step) const {
        return aligned(a) ? t - base >= 32 * step : t != base;
    }

    // starts the copies of tile t into dst; returns the mask of the tokens the row sees
    __device__ __forceinline__ uint32_t copy(const AttentionArgs& a, int hk, const Request& q, int t, int step, uint32_t dst, int lane,
                                             bool& bad) const {
        const int real_chunks = a.cache.dim * kBytes / 16;
        const char* kp = static_cast<const char*>(a.cache.k) + hk * a.cache.k_head * kBytes;
        const char* vp = static_cast<const char*>(a.cache.v) + hk * a.cache.v_head * kBytes;
        uint32_t mask;
        if (aligned(a)) {
            const int from = (t - base) / step;
            int64_t block = __shfl_sync(0xFFFFFFFFu, id, from);
            const int first = __shfl_sync(0xFFFFFFFFu, place, from);
            const int token = (q.tile0 + t) * kTile;
            mask = q.len - token < kTile ? (1u << (q.len - token)) - 1u : 0xFFFFu;
            if (q.start > token) mask &= 0xFFFFu << (q.start - token);
            if (block < 0 || block >= a.cache.blocks) {
                bad = true;
                mask = 0u;
                block = 0;
            }
            kp += (block * a.cache.k_block + first * a.cache.k_token) * kBytes;
            vp += (block * a.cache.v_block + first * a.cache.v_token) * kBytes;
            const int64_t ks = a.cache.k_token * kBytes, vs = a.cache.v_token * kBytes;
#pragma unroll
            for (int i = 0; i < kTile * CH / 32; ++i) {
                const int row = (i * 32 + lane) / CH, ch = (i * 32 + lane) % CH;
                const bool ok = (mask >> row) & 1u;
                if (ch < real_chunks) {
                    const uint32_t at = dst + tile_offset<CH>(row, ch);
                    cp_async_16_zfill(at, kp + row * ks + ch * 16, ok);
                    cp_async_16_zfill(at + kTile * Sh::kRowBytes, vp + row * vs + ch * 16, ok);
                }
            }
        } else {
            const bool valid = id >= 0 && id < a.cache.blocks;
            bad |= id != -1 && !valid;
            mask = __ballot_sync(0xFFFFFFFFu, valid) & 0xFFFFu;
            const int64_t block = valid ? id : 0, first = valid ? place : 0;
            const int64_t ko = (block * a.cache.k_block + first * a.cache.k_token) * kBytes;
            const int64_t vo = (block * a.cache.v_block + first * a.cache.v_token) * kBytes;
#pragma unroll
            for (int i = 0; i < kTile * CH / 32; ++i) {
                const int row = (i * 32 + lane) / CH, ch = (i * 32 + lane) % CH;
                const int64_t kr = __shfl_sync(0xFFFFFFFFu, ko, row);
                const int64_t vr = __shfl_sync(0xFFFFFFFFu, vo, row);
                const bool ok = (mask >> row) & 1u;
                if (ch < real_chunks) {
                    const uint32_t at = dst + tile_offset<CH>(row, ch);
                    cp_async_16_zfill(at, kp + kr + ch * 16, ok);
                    cp_async_16_zfill(at + kTile * Sh::kRowBytes, vp + vr + ch * 16, ok);
                }
            }
        }
        return mask;
    }
};

// Columns of a ring past dim are never copied: zeroed once.
__device__ __forceinline__ void clear_ring(uint8_t* smem, int bytes, int thread, int threads) {
    for (int i = thread; i < bytes / 16; i += threads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// The tiles [t0, t1) of one row, and where the row begins among all costs.
struct Segment {
    int at, b, row, t0, t1;
    Request q;
};

template <bool E4M3, int DP, int NT>
__global__ void __launch_bounds__((AttnShape<E4M3, DP, NT>::kShareWarps * 32), 1)
    k_attention_shares(const AttentionArgs a, const JoinPlan jp) {
    using Sh = AttnShape<E4M3, DP, NT>;
    constexpr int S = Sh::kStages, HEADS = Sh::kHeads, W = Sh::kShareWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t tile_mask[W][S];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int worker = blockIdx.x * W + warp;
    const uint32_t ring = smem_addr(smem) + warp * S * Sh::kStageBytes;
    const int rows = jp.rows;
    bool bad = false;

    if (a.cache.dim != DP) {
        clear_ring(smem, Sh::kSmem, threadIdx.x, W * 32);
        __syncthreads();
    }
    grid_dependency_wait();
    grid_dependents_launch();

    // --- the share of the warp ----------------------------------------------
    // Every warp forms the costs of all requests itself, kScan of them at a
    // time (lane i: kPer in a row from kPer * i on).  They fit 32 bits.
    constexpr int kPer = 4, kScan = 32 * kPer;
    int cost[kPer];  // of this lane's requests
    // the costs of requests base .. base + kScan - 1; returns those before this lane's, `sum`: all
    auto scan = [&](int base, int& sum) -> int {
        int own = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = base + lane * kPer + i;
            const int n = b < a.B ? request_of(a, b, bad).tiles : 0;
            cost[i] = n ? (n + kRowCost) * rows : 0;
            own += cost[i];
        }
        int inc = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d) inc += v;
        }
        sum = __shfl_sync(0xFFFFFFFFu, inc, 31);
        return inc - own;
    };
    int total = 0, head_start = 0;  // head_start: before this lane's requests, where one scan has all
    if (a.B <= kScan) {
        head_start = scan(0, total);
    } else {
#pragma unroll 8
        for (int b = lane; b < a.B; b += 32) {
            const int n = request_of(a, b, bad).tiles;
            total += n ? (n + kRowCost) * rows : 0;
        }
#pragma unroll
        for (int d = 16; d; d /= 2) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    }
    // requests without tokens
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (request_of(a, b, bad).tiles > 0) continue;
        store_empty(a, b, 0, a.q_heads, threadIdx.x, W * 32);
        if (jp.by_row)
            for (int i = threadIdx.x; i < rows; i += W * 32) jp.joins[b * rows + i] = make_int4(-1, 0, 0, 0);
    }
    int workers = min((total + kMinCost - 1) / kMinCost, jp.warps);
    // one request: rows of one length, so a multiple of them splits none unevenly
    if (a.B == 1 && workers > rows) workers -= workers % rows;
    if (!jp.by_row && lane == 0) jp.joins[worker] = make_int4(-1, 0, 0, 0);
    if (worker >= workers) {
        if (bad) raise_device_error(a.err, W4A16_DEVERR_SLOT);
        return;
    }
    // costs before worker i: equal shares, the remainder to the first ones
    const unsigned share = static_cast<unsigned>(total) / static_cast<unsigned>(workers), extra = total - share * workers;
    const int u0 = worker * share + min(static_cast<unsigned>(worker), extra);
    const int u1 = u0 + share + (worker < static_cast<int>(extra) ? 1 : 0);
    auto worker_of = [&](int u) -> int {
        const int big = extra * (share + 1);
        return u < big ? static_cast<unsigned>(u) / (share + 1) : extra + static_cast<unsigned>(u - big) / share;
    };
    // the request that holds the place u < total, and the costs before it
    auto locate = [&](int u, int& found_b, int& found_at) -> bool {
        int before = 0;
        for (int base = 0; base < a.B; base += kScan) {
            int sum = 0, start = head_start;
            if (a.B > kScan) start = scan(base, sum);
            start += before;
            int hit = -1;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (u >= start && u < start + cost[i]) {
                    hit = base + lane * kPer + i;
                    found_at = start;
                }
                start += cost[i];
            }
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, hit >= 0);
            if (who) {
                found_b = __shfl_sync(0xFFFFFFFFu, hit, __ffs(who) - 1);
                found_at = __shfl_sync(0xFFFFFFFFu, found_at, __ffs(who) - 1);
                return true;
            }
            before += sum;
        }
        return false;
    };

    // --- the rows of a share, in order ---------------------------------------
    auto open_segment = [&](Segment& s) {
        const int first = s.at + kRowCost;  // of the row's tiles
        s.t0 = max(u0 - first, 0);
        s.t1 = min(u1 - first, s.q.tiles);  // at most t0: nothing
    };
    auto next_segment = [&](Segment& s) -> bool {
        s.at += s.q.tiles + kRowCost;
        if (s.at + kRowCost >= u1) return false;
        if (++s.row == rows) {
            s.row = 0;
            do {
                if (++s.b >= a.B) return false;
                s.q = request_of(a, s.b, bad);
            } while (s.q.tiles == 0);
        }
        open_segment(s);
        return true;
    };
    Segment seg{};
    bool live = u1 > u0 && locate(u0, seg.b, seg.at);
    if (live) {
        seg.q = request_of(a, seg.b, bad);
        seg.row = static_cast<unsigned>(u0 - seg.at) / static_cast<unsigned>(seg.q.tiles + kRowCost);
        seg.at += seg.row * (seg.q.tiles + kRowCost);
        open_segment(seg);
        live = seg.t1 > seg.t0;
    }

    // The copies run ahead of the products: `ahead` is the segment of the next
    // tile to copy, ahead_t the tile.
    RowMath<E4M3, DP, NT> math;
    TileCopy<E4M3, DP, NT> copy;
    Segment ahead = seg;
    int ahead_t = seg.t0, ahead_hk = heads_of<HEADS>(a, seg.row).hk;
    bool more = live;
    if (more) copy.look_up(a, ahead.b, ahead.q, ahead_t, ahead.t1, 1, lane);
    // One step of the loop copies a tile and, once the ring is full, works on
    // the oldest one.
    int t = seg.t0, put = 0, slot = 0, primed = 0;
    bool fresh = true;  // the next tile is the first of its row here
    Heads hd{};
    while (live) {
        if (fresh) {
            // the queries are requested before the tiles, which they would queue behind
            fresh = false;
            hd = heads_of<HEADS>(a, seg.row);
            math.begin(a, seg.b, hd, lane);
            // and those of the row after this one brought to L2
            const int after_b = seg.row + 1 < rows ? seg.b : seg.b + 1;
            if (after_b < a.B) {
                const Heads h = heads_of<HEADS>(a, seg.row + 1 < rows ? seg.row + 1 : 0);
                constexpr int kLines = (DP + 63) / 64;
                for (int i = lane; i < h.n * kLines; i += 32)
                    if ((i % kLines) * 64 < a.cache.dim)
                        prefetch_l2(a.q + after_b * a.q_request + (h.first + i / kLines) * a.q_head + (i % kLines) * 64);
            }
        }
        const bool full = primed == S - 1;
        if (full) cp_async_wait_group<S - 2>();
        __syncwarp();
        if (more) {
            const uint32_t mask = copy.copy(a, ahead_hk, ahead.q, ahead_t, 1, ring + put * Sh::kStageBytes, lane, bad);
            if (lane == 0) tile_mask[warp][put] = mask;
            bool look = false;
            if (++ahead_t >= ahead.t1) {
                more = look = next_segment(ahead);
                ahead_t = ahead.t0;
                ahead_hk = heads_of<HEADS>(a, ahead.row).hk;
            }
            if (more && (look || copy.wants(a, ahead_t, 1))) copy.look_up(a, ahead.b, ahead.q, ahead_t, ahead.t1, 1, lane);
        }
        cp_async_commit();
        put = put + 1 == S ? 0 : put + 1;
        if (!full) {
            ++primed;
            continue;
        }
        if (t == seg.t0) math.ready(a, hd.hk, lane);
        math.tile(ring + slot * Sh::kStageBytes, tile_mask[warp][slot], lane);
        slot = slot + 1 == S ? 0 : slot + 1;
        if (++t < seg.t1) continue;

        math.reduce();
        const bool begins = seg.t0 == 0, ends = seg.t1 == seg.q.tiles;
        if (begins && ends) {
            math.finish(a, seg.b, hd, lane);
        } else {
            float* part = jp.part + (static_cast<int64_t>(worker) * 2 + (begins ? 1 : 0)) * Sh::kPartFloats;
            math.store_part(part, part + HEADS * DP, part + HEADS * (DP + 1), lane);
        }
        // a row that begins here: what the join launch has to do for it
        if (begins && lane == 0 && (jp.by_row || !ends))
            jp.joins[jp.by_row ? seg.b * rows + seg.row : worker] =
                ends ? make_int4(-1, 0, 0, 0) : make_int4(seg.b, seg.row, worker, worker_of(seg.at + kRowCost + seg.q.tiles - 1));
        live = next_segment(seg);
        t = seg.t0;
        fresh = true;
    }
    cp_async_wait_group<0>();
    if (bad) raise_device_error(a.err, W4A16_DEVERR_SLOT);
}

// Where the CTA `rank` of the cluster has what this one has at `local`.
__device__ __forceinline__ uint32_t cluster_address(const void* local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    return remote;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t at) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

template <bool E4M3>
__device__ __forceinline__ void store_lse(const AttentionArgs& a, int b, const Heads& hd, int h, float m, float l) {
    if (a.lse && h < hd.n) a.lse[static_cast<int64_t>(b) * a.q_heads + hd.first + h] = lse_of<E4M3>(m, l);
}

// The factors of up to eight parts of a head, one lane each (lanes 8 h .. 8 h + 7
// of a warp); m and l become those of all parts.
__device__ __forceinline__ float join_factor(float& m, float& l) {
    float top = m, all;
#pragma unroll
    for (int d = 1; d < 8; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));  // of an empty part: -infinity
    const float f = l != 0.f ? part_factor(m, top) : 0.f;
    all = l * f;
#pragma unroll
    for (int d = 1; d < 8; d *= 2) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
    m = top, l = all;
    return f;
}
__device__ __forceinline__ void add_scaled(float4& o, const float4& x, float2 f) {
    o.x = fmaf(x.x, f.x, o.x), o.y = fmaf(x.y, f.y, o.y);
    o.z = fmaf(x.z, f.x, o.z), o.w = fmaf(x.w, f.y, o.w);
}

// A part's 16 dims of 8 heads, with what joining them takes: m and l of the
// lane's two heads.
struct DimPart {
    float4 o;
    float m[2], l[2];
    __device__ __forceinline__ void clear() {
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ __forceinline__ void add(const float4& x, float2 xm, float2 xl) {
        const float pm[2] = {xm.x, xm.y}, pl[2] = {xl.x, xl.y};
        float f0[2], f1[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float top = pl[e] != 0.f ? fmaxf(m[e], pm[e]) : m[e];
            f0[e] = part_factor(m[e], top);
            f1[e] = pl[e] != 0.f ? part_factor(pm[e], top) : 0.f;
            m[e] = top;
            l[e] = l[e] * f0[e] + pl[e] * f1[e];
        }
        o.x = o.x * f0[0] + x.x * f1[0], o.y = o.y * f0[1] + x.y * f1[1];
        o.z = o.z * f0[0] + x.z * f1[0], o.w = o.w * f0[1] + x.w * f1[1];
    }
    // the result: dims of step k, heads of block n
    template <bool E4M3>
    __device__ __forceinline__ void finish(const AttentionArgs& a, int b, const Heads& hd, int n, int k, int lane) const {
        const int r = lane >> 2, c = lane & 3;
        const float vs = E4M3 ? a.cache.v_scale[hd.hk] : 1.f;
        const float f0 = l[0] != 0.f ? vs / l[0] : 0.f, f1 = l[1] != 0.f ? vs / l[1] : 0.f;
        const bool have = n * 8 + r < hd.n && k * 16 < a.cache.dim;
        uint16_t* out = a.out + b * a.out_request + (hd.first + n * 8 + r) * a.out_head + k * 16;
        store_dims<E4M3>(o, f0, f1, have ? out : nullptr, c);
        if (k == 0 && r == 0) {
            store_lse<E4M3>(a, b, hd, n * 8 + 2 * c, m[0], l[0]);
            store_lse<E4M3>(a, b, hd, n * 8 + 2 * c + 1, m[1], l[1]);
        }
    }
};

// Joins the parts of a row: grid (row, slice of its accumulators); threads
// (x: accumulators, y: group, of which each takes every n-th part, so that
// many parts are on their way at once).
constexpr int kJoinThreads = 512;  // at most
constexpr int kJoinDepth = 3;  // parts a thread requests together

template <bool E4M3, int DP, int NT>
__global__ void __launch_bounds__(kJoinThreads) k_attention_join(const AttentionArgs a, const JoinPlan jp) {
    using Sh = AttnShape<E4M3, DP, NT>;
    constexpr int HEADS = Sh::kHeads, KS = Sh::kSteps;
    __shared__ DimPart sums[kJoinThreads / 2];
    grid_dependents_launch();
    grid_dependency_wait();
    const int4 d = __ldcg(jp.joins + blockIdx.x);
    if (d.x < 0) return;
    const int unit = blockIdx.y * blockDim.x + threadIdx.x;  // accumulator: (head block n, step k, lane)
    const int lane = unit & 31, k = (unit >> 5) % KS, n = (unit >> 5) / KS, c = lane & 3;
    DimPart s;
    s.clear();
#pragma unroll 1
    for (int q = d.z + static_cast<int>(threadIdx.y); q <= d.w; q += blockDim.y * kJoinDepth) {
        float4 o[kJoinDepth];
        float2 m[kJoinDepth], l[kJoinDepth];
#pragma unroll
        for (int i = 0; i < kJoinDepth; ++i) {
            const int p = q + i * blockDim.y;
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            m[i] = l[i] = make_float2(0.f, 0.f);
            if (p <= d.w) {
                const float* part = jp.part + (static_cast<int64_t>(p) * 2 + (p == d.z ? 1 : 0)) * Sh::kPartFloats;
                o[i] = __ldcg(reinterpret_cast<const float4*>(part) + unit);
                m[i] = __ldcg(reinterpret_cast<const float2*>(part + HEADS * DP) + n * 4 + c);
                l[i] = __ldcg(reinterpret_cast<const float2*>(part + HEADS * (DP + 1)) + n * 4 + c);
            }
        }
#pragma unroll
        for (int i = 0; i < kJoinDepth; ++i) s.add(o[i], m[i], l[i]);
    }
    // the groups, pairwise (one after another, sixteen took 2.2 us)
#pragma unroll 1
    for (int half = static_cast<int>(blockDim.y) / 2; half >= 1; half /= 2) {
        const int g = threadIdx.y;
        if (g >= half && g < 2 * half) sums[(g - half) * blockDim.x + threadIdx.x] = s;
        __syncthreads();
        if (g < half) {
            const DimPart& x = sums[g * blockDim.x + threadIdx.x];
            s.add(x.o, make_float2(x.m[0], x.m[1]), make_float2(x.l[0], x.l[1]));
        }
        __syncthreads();
    }
    if (threadIdx.y > 0) return;
    s.finish<E4M3>(a, d.x, heads_of<HEADS>(a, d.y), n, k, lane);
}

// kRowWarps / wpr rows per CTA, wpr warps for each; or (cluster > 1, wpr =
// kRowWarps) a row per cluster.  Tiles go round the CTAs of a row, then their
// warps.
template <bool E4M3, int DP, int NT>
__global__ void __launch_bounds__((AttnShape<E4M3, DP, NT>::kRowWarps * 32), 1)
    k_attention_rows(const AttentionArgs a, const int rows, const int wpr, const int cluster) {
    using Sh = AttnShape<E4M3, DP, NT>;
    constexpr int S = Sh::kRowStages, HEADS = Sh::kHeads, KS = Sh::kSteps, W = Sh::kRowWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t tile_mask[W][S];
    __shared__ __align__(8) float part_m[W][HEADS], part_l[W][HEADS], part_f[W][HEADS], cta_m[HEADS], cta_l[HEADS], cta_f[8][HEADS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int wir = warp & (wpr - 1), warp0 = warp - wir;  // warp in its row (of this CTA), and the row's first
    const int first_tile = wir * cluster + rank, step = wpr * cluster;
    const uint32_t ring = smem_addr(smem) + warp * Sh::kRowRing;
    const unsigned id = cluster > 1 ? blockIdx.x / static_cast<unsigned>(cluster) : (blockIdx.x * W + warp) / static_cast<unsigned>(wpr);
    const int b = static_cast<int>(id / static_cast<unsigned>(rows)), row = static_cast<int>(id - b * static_cast<unsigned>(rows));
    bool bad = false;
    if (a.cache.dim != DP) {
        clear_ring(smem, Sh::kRowSmem, threadIdx.x, W * 32);
        __syncthreads();
    }
    const Heads hd = b < a.B ? heads_of<HEADS>(a, row) : Heads{};
    grid_dependency_wait();
    grid_dependents_launch();
    // Queries, block ids (where they do not depend on the length) and length are
    // requested together.
    RowMath<E4M3, DP, NT> math;
    TileCopy<E4M3, DP, NT> copy;
    Request q{};
    if (b < a.B) {
        const bool early = a.window == 0 && TileCopy<E4M3, DP, NT>::aligned(a);
        if (early) copy.look_up(a, b, q, first_tile, (a.most + kTile - 1) / kTile, step, lane);
        math.begin(a, b, hd, lane);
        q = request_of(a, b, bad);
        if (!early) copy.look_up(a, b, q, first_tile, q.tiles, step, lane);
        if (q.tiles == 0 && rank == 0) store_empty(a, b, hd.first, hd.n, wir * 32 + lane, wpr * 32);
    }
    if (first_tile < q.tiles) {
        int ahead = first_tile, put = 0, slot = 0, primed = 0;
        for (int t = first_tile; t < q.tiles;) {
            const bool full = primed == S - 1;
            if (full) cp_async_wait_group<S - 2>();
            __syncwarp();
            if (ahead < q.tiles) {
                const uint32_t mask = copy.copy(a, hd.hk, q, ahead, step, ring + put * Sh::kStageBytes, lane, bad);
                if (lane == 0) tile_mask[warp][put] = mask;
                ahead += step;
                if (ahead < q.tiles && copy.wants(a, ahead, step)) copy.look_up(a, b, q, ahead, q.tiles, step, lane);
            }
            cp_async_commit();
            put = put + 1 == S ? 0 : put + 1;
            if (!full) {
                ++primed;
                continue;
            }
            if (t == first_tile) math.ready(a, hd.hk, lane);
            math.tile(ring + slot * Sh::kStageBytes, tile_mask[warp][slot], lane);
            slot = slot + 1 == S ? 0 : slot + 1;
            t += step;
        }
        cp_async_wait_group<0>();
        __syncwarp();
        math.reduce();
        if (step == 1 || q.tiles == 1) {  // nobody else has a part
            math.finish(a, b, hd, lane);
        } else {
            math.store_part(reinterpret_cast<float*>(smem + warp * Sh::kRowRing), part_m[warp], part_l[warp], lane);
        }
    }
    if (bad) raise_device_error(a.err, W4A16_DEVERR_SLOT);
    if (step == 1) return;
    __syncthreads();
    const bool joins = q.tiles > 1;
    const int used = min((q.tiles - rank + cluster - 1) / cluster, wpr);  // warps here that had a tile (at most 0: none)
    const int r = lane >> 2, c = lane & 3;
    const float vs = E4M3 && joins ? a.cache.v_scale[hd.hk] : 1.f;
    float4* const cta_part = reinterpret_cast<float4*>(smem + Sh::kPartBytes);
    if (joins)
        for (int x = wir * 32 + lane; x < HEADS * 8; x += wpr * 32) {
            const int h = x >> 3, i = x & 7;
            float m = -INFINITY, l = 0.f;
            if (i < used) m = part_m[warp0 + i][h], l = part_l[warp0 + i][h];
            const float f = join_factor(m, l);
            if (i < wpr) part_f[warp0 + i][h] = f;
            if (i == 0) {
                if (cluster == 1) {
                    store_lse<E4M3>(a, b, hd, h, m, l);
                    part_l[warp0][h] = l != 0.f ? vs / l : 0.f;  // now the result's factor
                } else {
                    cta_m[h] = m, cta_l[h] = l;
                }
            }
        }
    __syncthreads();
    if (!joins) return;
#pragma unroll 1
    for (int u = wir; u < NT * KS; u += wpr) {
        const int n = u / KS, k = u % KS, h = n * 8 + 2 * c;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < used; ++i)
            add_scaled(o, reinterpret_cast<const float4*>(smem + (warp0 + i) * Sh::kRowRing)[u * 32 + lane],
                       *reinterpret_cast<const float2*>(&part_f[warp0 + i][h]));
        if (cluster == 1) {
            const float2 f = *reinterpret_cast<const float2*>(&part_l[warp0][h]);
            uint16_t* out = a.out + b * a.out_request + (hd.first + n * 8 + r) * a.out_head + k * 16;
            store_dims<E4M3>(o, f.x, f.y, n * 8 + r < hd.n && k * 16 < a.cache.dim ? out : nullptr, c);
        } else {
            cta_part[u * 32 + lane] = o;
        }
    }
    if (cluster == 1) return;
    cluster_barrier();
    for (int x = threadIdx.x; x < HEADS * 8; x += W * 32) {
        const int h = x >> 3, i = x & 7;
        float m = -INFINITY, l = 0.f;
        if (i < cluster) m = ld_cluster_f32(cluster_address(&cta_m[h], i)), l = ld_cluster_f32(cluster_address(&cta_l[h], i));
        cta_f[i][h] = join_factor(m, l);
        if (i == 0) {
            if (rank == 0) store_lse<E4M3>(a, b, hd, h, m, l);
            part_l[0][h] = l != 0.f ? vs / l : 0.f;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int u = warp * cluster + rank; u < NT * KS; u += W * cluster) {
        const int n = u / KS, k = u % KS, h = n * 8 + 2 * c;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < cluster; ++i)
            add_scaled(o, ld_cluster_f32x4(cluster_address(cta_part + u * 32 + lane, i)), *reinterpret_cast<const float2*>(&cta_f[i][h]));
        const float2 f = *reinterpret_cast<const float2*>(&part_l[0][h]);
        uint16_t* out = a.out + b * a.out_request + (hd.first + n * 8 + r) * a.out_head + k * 16;
        store_dims<E4M3>(o, f.x, f.y, n * 8 + r < hd.n && k * 16 < a.cache.dim ? out : nullptr, c);
    }
    cluster_barrier();  // nobody leaves while its part may be read
}

// early: the grid's CTAs may start while the preceding one runs (they wait for its end themselves)
template <class... Params, class... Args>
cudaError_t launch_kernel(void (*kernel)(Params...), bool early, int cluster, dim3 grid, dim3 block, int smem, cudaStream_t s,
                          Args... args) {
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e == cudaSuccess) e = ensure_shared_carveout(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool E4M3, int DP, int NT>
cudaError_t launch_attention_shape(const AttentionArgs& all, const DeviceInfo& dev, JoinPlan jp, cudaStream_t s) {
    using Sh = AttnShape<E4M3, DP, NT>;
    AttentionArgs a = all;
    jp.rows = rows_of_request(a.q_heads, a.cache.heads, Sh::kHeads);
    int64_t all_rows = static_cast<int64_t>(a.B) * jp.rows;
    const int tiles = most_tiles(a.most, a.window);  // of a row
    // short rows: as many warps for each as one wave of CTAs has, if that leaves
    // a warp few tiles
    {
        constexpr int W = Sh::kRowWarps;
        int wpr = W, cluster = 1;
        while (wpr > 1 && all_rows * wpr > static_cast<int64_t>(dev.sms) * W) wpr /= 2;
        // (19 tiles of 8 rows: 6.2 us with a CTA each, 6.9 with two, 5.9 with four)
        if (Sh::kClusters && wpr == W && tiles > kRowEnough * W)
            while (cluster < 8 && tiles > W * cluster && all_rows * cluster * 2 <= dev.sms) cluster *= 2;
        while (cluster > 1 && max_active_clusters(reinterpret_cast<const void*>(k_attention_rows<E4M3, DP, NT>), W * 32,
                                                  Sh::kRowSmem, cluster) < all_rows)
            cluster /= 2;
        const int64_t grid = cluster > 1 ? all_rows * cluster : (all_rows * wpr + W - 1) / W;
        if (tiles <= kRowTiles * wpr * cluster)
            return launch_kernel(k_attention_rows<E4M3, DP, NT>, true, cluster, dim3(static_cast<unsigned>(grid)), dim3(W * 32),
                                 Sh::kRowSmem, s, a, jp.rows, wpr, cluster);
    }
    const int ctas = std::min(dev.sms, most_workers(DP) / Sh::kShareWarps);
    jp.warps = ctas * Sh::kShareWarps;
    // as many requests at a time as have costs of 32 bits (one has: attention_costs_fit)
    const int64_t fit = kMostCost / (static_cast<int64_t>(tiles + kRowCost) * jp.rows);
    for (int from = 0; from < all.B; from += a.B) {
        a.B = static_cast<int>(std::min<int64_t>(all.B - from, fit));
        a.q = all.q + from * a.q_request, a.out = all.out + from * a.out_request;
        a.block_table = all.block_table + from * a.table_stride, a.kv_len = all.kv_len + from;
        a.lse = all.lse ? all.lse + static_cast<int64_t>(from) * a.q_heads : nullptr;
        all_rows = static_cast<int64_t>(a.B) * jp.rows;
        jp.by_row = all_rows <= jp.warps;
        // (early, because a CTA has an SM for itself: several smaller ones that are placed
        // around others leave holes in the register file, and those that no longer fit then
        // run when the rest are done -- 20 key/value heads of 64 dims, 24 requests: 26 us)
        cudaError_t e = launch_kernel(k_attention_shares<E4M3, DP, NT>, true, 1, dim3(ctas), dim3(Sh::kShareWarps * 32), Sh::kSmem,
                                      s, a, jp);
        if (e != cudaSuccess) return e;
        // few rows: their accumulators over several CTAs, down to a warp's; as many
        // groups as a row has parts for, if rows are alike
        const int places = jp.by_row ? static_cast<int>(all_rows) : jp.warps, units = Sh::kHeads * DP / 4;
        int width = 128;
        while (units % width || (width > 32 && places * (units / width) < dev.sms)) width /= 2;
        const int parts = jp.warps / places + 2;
        int groups = 1;
        while (groups * width < kJoinThreads && groups * kJoinDepth < parts) groups *= 2;
        e = launch_kernel(k_attention_join<E4M3, DP, NT>, true, 1, dim3(places, units / width), dim3(width, groups), 0, s, a, jp);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <bool E4M3>
cudaError_t launch_attention_type(const AttentionArgs& a, const DeviceInfo& dev, const JoinPlan& jp, cudaStream_t s) {
    const bool wide = a.q_heads / a.cache.heads > 8;
    // 16 heads of 256 dims fill a warp's registers: two rows of 8 are faster while the second
    // finds the cache in L2 (8 requests, windows of 4096: 15.4 us against 18.0; 134 MB over
    // e4m3 50 against 58; but 1.07 GB of bf16 328 against 216)
    const int64_t visible = a.window > 0 && a.window < a.most ? a.window : a.most;
    const bool in_l2 = static_cast<double>(a.B) * visible * a.cache.heads * a.cache.dim * (E4M3 ? 2 : 4) <= (1 << 27);
    switch (padded_dim(a.cache.dim)) {
        case 64: return wide ? launch_attention_shape<E4M3, 64, 2>(a, dev, jp, s) : launch_attention_shape<E4M3, 64, 1>(a, dev, jp, s);
        case 96: return wide ? launch_attention_shape<E4M3, 96, 2>(a, dev, jp, s) : launch_attention_shape<E4M3, 96, 1>(a, dev, jp, s);
        case 128: return wide ? launch_attention_shape<E4M3, 128, 2>(a, dev, jp, s) : launch_attention_shape<E4M3, 128, 1>(a, dev, jp, s);
        case 192: return wide ? launch_attention_shape<E4M3, 192, 2>(a, dev, jp, s) : launch_attention_shape<E4M3, 192, 1>(a, dev, jp, s);
        default: return wide && !in_l2 ? launch_attention_shape<E4M3, 256, 2>(a, dev, jp, s) : launch_attention_shape<E4M3, 256, 1>(a, dev, jp, s);
    }
}

}  // namespace
}  // namespace w4a16
