// Attention of one new token per request over a paged key/value cache
// (w4a16_paged_attention): the kernel, for one cache type per translation unit.
//
// A row is one request, one key/value head and up to 8 * NT of the query
// heads that share it.  For the tokens j a row sees,
//     s_j = c q . k_j (log2 units),  m = max s_j,  p_j = 2^(s_j - m),
//     l = sum p_j,  o = sum p_j v_j,  out = o / l,
// in one pass: a larger m scales the running l and o by 2^(m_old - m).
// Partial (m, l, o) of disjoint token sets join the same way, in any grouping.
//
// Bound by HBM: each key and value is read once, for 2 * heads operations a
// byte at most.  So the kernel is built around the copies:
//   - Work is dealt in tiles of 16 tokens, rows one after another, and every
//     warp takes an equal consecutive share of all tiles, whatever the lengths
//     are (each CTA forms the sum of the tile counts itself; a row counts a
//     tile more than it has, for its queries and its result).
//   - A warp works alone, through a ring of its own of cp.async stages that
//     runs on across rows; a row inside its share it finishes alone.  Only the
//     two rows at the ends of its share may be others' too: their parts meet
//     in shared memory once the CTA's warps are done, and what the CTA does
//     not hold whole goes to the workspace, for a second launch to join
//     (paged_attention.cu), always in the order of the tokens.
//   - The products run on the warp MMA with the keys as the 16-row operand
//     (tokens) and the heads as its 8 columns: one product covers 8 query
//     heads, and the transposed second product (values^T times p^T) takes the
//     probabilities from the accumulators by one 8x8 transpose in registers.
//     (tcgen05 would want 64 or more query rows; here there are 1 to 16.)
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "paged_attention.h"

namespace w4a16 {
namespace {

constexpr int kTile = 16;  // tokens of a tile: the MMA's rows
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kRowCost = 1;   // a row's queries and result, in tiles
constexpr int kMinCost = 4;   // a warp's share at least
constexpr int kWholeTiles = 32;  // rows that cannot be longer are not split over CTAs

// Shared memory: a ring of kStages tiles per warp, and a place for the (o) of
// the row a warp's share begins inside of (the row it ends inside of goes
// where its ring was).
template <bool E4M3, int DP, int NT>
struct AttnShape {
    static constexpr int kHeads = 8 * NT;
    static constexpr int kRowBytes = DP * (E4M3 ? 1 : 2);
    static constexpr int kChunks = kRowBytes / 16;             // 16-byte chunks of a row
    static constexpr int kStageBytes = 2 * kTile * kRowBytes;  // keys, then values
    static constexpr int kPartBytes = kHeads * DP * 4;
    static constexpr int kJoinBytes = kAttnWarps * kPartBytes;
    // two CTAs an SM with three or more stages where that fits, else one
    static constexpr int kTwo = (112 * 1024 - kJoinBytes) / (kAttnWarps * kStageBytes);
    static constexpr int kOne = (225 * 1024 - kJoinBytes) / (kAttnWarps * kStageBytes);
    static constexpr int kPerSm = kTwo >= 3 ? 2 : 1;
    static constexpr int kFit = kPerSm == 2 ? kTwo : kOne;
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kRingBytes = kStages * kStageBytes;  // of a warp
    static constexpr int kSmem = kAttnWarps * kRingBytes + kJoinBytes;
    static_assert(kStages >= 2 && kRingBytes >= kPartBytes + 3 * 2 * kAttnWarps * kHeads * 4, "ring too short");
};

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

// n / d for n >= 0, d > 0: in 32 bits where both fit, as they do in all but
// the largest calls (a 64-bit division takes about 200 ns here)
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
    if (((n | d) >> 32) == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
    return n / d;
}

// The tiles [t0, t1) of one row, and where the row begins among all costs.
struct Segment {
    int64_t at;
    int b, row, t0, t1;
    Request q;
};

// float index of (head h, dim d) in a part in shared memory: swizzled so that a
// fragment's 8 dims x 4 head pairs lie in different banks, four dims together
template <bool E4M3, int DP>
__device__ __forceinline__ int part_index(int h, int d) {
    return h * DP + (d ^ (((h >> 1) & 3) * (E4M3 ? 16 : 8)));
}

template <bool E4M3, int DP, int NT>
__global__ void __launch_bounds__(kAttnThreads) k_paged_attention_mma(const AttentionArgs a, const JoinPlan jp) {
    using Sh = AttnShape<E4M3, DP, NT>;
    constexpr int CH = Sh::kChunks, S = Sh::kStages, HEADS = Sh::kHeads, KS = DP / 16;
    constexpr int kBytes = E4M3 ? 1 : 2;
    constexpr float kBias = E4M3 ? kE4m3Bias : 0.f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t tile_mask[kAttnWarps][S];
    // parts of a warp: 0 of the row its share begins inside of, 1 of the one it ends inside of
    __shared__ int64_t part_at[kAttnWarps * 2];
    __shared__ int part_b[kAttnWarps * 2], part_row[kAttnWarps * 2], part_ends[kAttnWarps * 2], part_tiles[kAttnWarps * 2];
    __shared__ float part_m[kAttnWarps * 2][HEADS], part_l[kAttnWarps * 2][HEADS];
    __shared__ uint32_t part_members[kAttnWarps * 2];
    // once the rings are done, behind the first one's part: a part's factor, and the maximum and sum of its row
    using PartFloats = float[HEADS];
    PartFloats* const part_f = reinterpret_cast<PartFloats*>(smem + Sh::kPartBytes);
    PartFloats *const part_top = part_f + kAttnWarps * 2, *const part_all = part_top + kAttnWarps * 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * Sh::kRingBytes;
    auto part_of = [&](int i) -> float* {
        return reinterpret_cast<float*>(smem + ((i & 1) ? (i >> 1) * Sh::kRingBytes
                                                        : kAttnWarps * Sh::kRingBytes + (i >> 1) * Sh::kPartBytes));
    };
    const int D = a.cache.dim, G = a.q_heads / a.cache.heads;
    const int chunks_of_group = (G + HEADS - 1) / HEADS;
    const int rows = jp.rows;  // of a request
    const int real_chunks = D * kBytes / 16;
    bool bad = false;

    if (D != DP) {  // columns past dim are never copied: zero them once
        for (int i = threadIdx.x; i < kAttnWarps * Sh::kRingBytes / 16; i += kAttnThreads)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (threadIdx.x < kAttnWarps * 2) part_b[threadIdx.x] = -1;
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();

    // --- the share of each warp ---------------------------------------------
    // Every warp forms the costs of all requests itself, kScan of them at a
    // time (lane i: kPer in a row from kPer * i on): no barrier is needed.
    constexpr int kPer = 4, kScan = 32 * kPer;
    int64_t cost[kPer];  // of this lane's requests
    // the costs of requests base .. base + kScan - 1; returns those before this lane's, `sum`: all
    auto scan = [&](int base, int64_t& sum) -> int64_t {
        int64_t own = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = base + lane * kPer + i;
            const int n = b < a.B ? request_of(a, b, bad).tiles : 0;
            cost[i] = n ? static_cast<int64_t>(n + kRowCost) * rows : 0;
            own += cost[i];
        }
        int64_t inc = own;
#pragma unroll 1
        for (int d = 1; d < 32; d *= 2) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d) inc += v;
        }
        sum = __shfl_sync(0xFFFFFFFFu, inc, 31);
        return inc - own;
    };
    int64_t total = 0, head_start = 0;  // head_start: before this lane's, of the first kScan requests
    for (int base = 0; base < a.B; base += kScan) {
        int64_t sum;
        const int64_t start = scan(base, sum);
        if (base == 0) head_start = start;
        total += sum;
    }
    // requests without tokens
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (request_of(a, b, bad).tiles > 0) continue;
        for (int i = threadIdx.x; i < a.q_heads * (D / 8); i += kAttnThreads) {
            const int h = i / (D / 8), d = (i - h * (D / 8)) * 8;
            *reinterpret_cast<uint4*>(a.out + b * a.out_request + h * a.out_head + d) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (a.lse)
            for (int h = threadIdx.x; h < a.q_heads; h += kAttnThreads)
                a.lse[static_cast<int64_t>(b) * a.q_heads + h] = -INFINITY;
        if (jp.split && jp.by_row)
            for (int i = threadIdx.x; i < rows; i += kAttnThreads) jp.joins[b * rows + i] = make_int4(-1, 0, 0, 0);
    }
    const int64_t want = quotient(total + kMinCost * kAttnWarps - 1, kMinCost * kAttnWarps);
    int ctas = want < gridDim.x ? static_cast<int>(want) : static_cast<int>(gridDim.x);
    // one request: rows of one length, so a multiple of them splits none unevenly
    if (a.B == 1 && ctas > rows) ctas -= ctas % rows;
    if (static_cast<int>(blockIdx.x) >= ctas) {
        if (jp.split && !jp.by_row && threadIdx.x == 0) jp.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
        if (bad) raise_device_error(a.err, W4A16_DEVERR_SLOT);
        return;
    }
    // costs before CTA i: equal shares, the remainder to the first ones
    const int64_t share = quotient(total, ctas), extra = total - share * ctas;
    auto cta_begin = [&](int i) { return i * share + (i < extra ? i : extra); };
    auto cta_of = [&](int64_t u) {
        const int64_t big = extra * (share + 1);
        return static_cast<int>(u < big ? quotient(u, share + 1) : extra + quotient(u - big, share));
    };
    // the request that holds the place u < total, and the costs before it
    auto locate = [&](int64_t u, int& found_b, int64_t& found_at) -> bool {
        int64_t before = 0;
        for (int base = 0; base < a.B; base += kScan) {
            int64_t sum = 0, start = head_start;
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
    int64_t begin = cta_begin(blockIdx.x), end = cta_begin(blockIdx.x + 1);
    int first_b = 0;
    int64_t first_at = 0;
    if (!jp.split) {
        // whole rows: from the first that begins in the share to the last that does
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            int64_t& u = i ? end : begin;
            if (u >= total || !locate(u, first_b, first_at)) continue;
            const int n = request_of(a, first_b, bad).tiles + kRowCost;
            u = first_at + quotient(u - first_at + n - 1, n) * n;
        }
    }
    static_assert(kAttnWarps == 4, "shares of four warps");
    const int64_t u0 = begin + ((end - begin) * warp >> 2), u1 = begin + ((end - begin) * (warp + 1) >> 2);

    // --- the rows of a share, in order ---------------------------------------
    auto open_segment = [&](Segment& s) {
        const int64_t first = s.at + kRowCost;  // of the row's tiles
        s.t0 = u0 > first ? static_cast<int>(u0 - first) : 0;
        s.t1 = u1 - first < s.q.tiles ? static_cast<int>(u1 - first) : s.q.tiles;  // at most t0: nothing
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
    bool live = u1 > u0 && locate(u0, first_b, first_at);
    if (live) {
        seg.b = first_b;
        seg.q = request_of(a, seg.b, bad);
        seg.row = static_cast<int>(quotient(u0 - first_at, seg.q.tiles + kRowCost));
        seg.at = first_at + static_cast<int64_t>(seg.row) * (seg.q.tiles + kRowCost);
        open_segment(seg);
        live = seg.t1 > seg.t0;
    }

    // The copies run ahead of the products: `ahead` is the segment of the next
    // tile to copy, ahead_t the tile.  Block ids are loaded early: where a tile
    // lies in one block, those of 32 tiles at once (lane i: tile win_t + i),
    // else those of the next tile's tokens (lanes i and i + 16: token i).
    Segment ahead = seg;
    int ahead_t = seg.t0, win_t = seg.t0 - 32;
    bool more = live;
    int ahead_id = -1, ahead_place = 0;
    const bool aligned_pages = a.cache.page % kTile == 0;
    auto settle = [&]() {
        if (more && ahead_t >= ahead.t1) {
            more = next_segment(ahead);
            ahead_t = ahead.t0;
            win_t = ahead_t - 32;
        }
        if (!more || (aligned_pages && ahead_t < win_t + 32)) return;
        win_t = ahead_t;
        const int token = aligned_pages ? (ahead.q.tile0 + ahead_t + lane) * kTile
                                        : (ahead.q.tile0 + ahead_t) * kTile + (lane & 15);
        const int col = static_cast<int>(static_cast<unsigned>(token) / static_cast<unsigned>(a.cache.page));
        ahead_place = token - col * a.cache.page;
        ahead_id = -1;
        if (aligned_pages ? ahead_t + lane < ahead.t1 : token >= ahead.q.start && token < ahead.q.len) {
            ahead_id = a.block_table[ahead.b * a.table_stride + col];
            if (ahead_id < 0) ahead_id = -2;
        }
    };
    auto copy_tile = [&](int slot) {
        if (more) {
            const int hk = ahead.row / chunks_of_group;
            const char* kp = static_cast<const char*>(a.cache.k) + hk * a.cache.k_head * kBytes;
            const char* vp = static_cast<const char*>(a.cache.v) + hk * a.cache.v_head * kBytes;
            const uint32_t dst = ring + slot * Sh::kStageBytes;
            uint32_t mask;  // the tokens of the tile that the row sees
            if (aligned_pages) {
                int64_t id = __shfl_sync(0xFFFFFFFFu, ahead_id, ahead_t - win_t);
                const int place = __shfl_sync(0xFFFFFFFFu, ahead_place, ahead_t - win_t);
                const int token = (ahead.q.tile0 + ahead_t) * kTile;
                mask = ahead.q.len - token < kTile ? (1u << (ahead.q.len - token)) - 1u : 0xFFFFu;
                if (ahead.q.start > token) mask &= 0xFFFFu << (ahead.q.start - token);
                if (id < 0 || id >= a.cache.blocks) {
                    bad = true;
                    mask = 0u;
                    id = 0;
                }
                kp += (id * a.cache.k_block + place * a.cache.k_token) * kBytes;
                vp += (id * a.cache.v_block + place * a.cache.v_token) * kBytes;
                const int64_t kt = a.cache.k_token * kBytes, vt = a.cache.v_token * kBytes;
#pragma unroll
                for (int i = 0; i < kTile * CH / 32; ++i) {
                    const int row = (i * 32 + lane) / CH, ch = (i * 32 + lane) % CH;
                    const bool ok = (mask >> row) & 1u;
                    if (ch < real_chunks) {
                        const uint32_t at = dst + tile_offset<CH>(row, ch);
                        cp_async_16_zfill(at, kp + row * kt + ch * 16, ok);
                        cp_async_16_zfill(at + kTile * Sh::kRowBytes, vp + row * vt + ch * 16, ok);
                    }
                }
            } else {
                const bool valid = ahead_id >= 0 && ahead_id < a.cache.blocks;
                bad |= ahead_id != -1 && !valid;
                mask = __ballot_sync(0xFFFFFFFFu, valid) & 0xFFFFu;
                const int64_t id = valid ? ahead_id : 0, place = valid ? ahead_place : 0;
                const int64_t ko = (id * a.cache.k_block + place * a.cache.k_token) * kBytes;
                const int64_t vo = (id * a.cache.v_block + place * a.cache.v_token) * kBytes;
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
            if (lane == 0) tile_mask[warp][slot] = mask;
            ++ahead_t;
            settle();
        }
        cp_async_commit();
    };

    settle();
    // One step of the loop copies a tile and, once the ring is full, works on
    // the oldest one.
    int t = seg.t0, put = 0, slot = 0, primed = 0;
    bool fresh = true;  // the next tile is the first of its row here
    int hk = 0, head0 = 0, heads = 0;  // key/value head, first query head and their number
    uint32_t qf[NT][KS][2];            // queries as B fragments (columns: heads)
    float sl[NT][2];                   // score scale of columns 2c, 2c + 1
    float m[NT][2], l[NT][2], o[NT][KS][4];
    while (live) {
        if (fresh) {
            // the queries are requested before the tiles, which they would queue behind
            fresh = false;
            hk = seg.row / chunks_of_group;
            const int chunk = seg.row - hk * chunks_of_group;
            head0 = hk * G + chunk * HEADS;
            heads = min(HEADS, G - chunk * HEADS);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint16_t* qp = a.q + seg.b * a.q_request + (head0 + n * 8 + r) * a.q_head;
                const bool have = n * 8 + r < heads;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    qf[n][k][0] = qf[n][k][1] = 0u;
                    if (have && k * 16 < D) {
                        // bf16: dims 2c, 2c + 1 and 8 further; e4m3: the four dims whose codes one word holds
                        const int d = k * 16 + (E4M3 ? 4 * c : 2 * c);
                        qf[n][k][0] = *reinterpret_cast<const uint32_t*>(qp + d);
                        qf[n][k][1] = *reinterpret_cast<const uint32_t*>(qp + d + (E4M3 ? 2 : 8));
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[n][e] = -INFINITY;
                    l[n][e] = 0.f;
                }
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][k][e] = 0.f;
            }
            // and those of the row after this one brought to L2
            const int after_b = seg.row + 1 < rows ? seg.b : seg.b + 1, after_row = seg.row + 1 < rows ? seg.row + 1 : 0;
            if (after_b < a.B) {
                const int g = after_row / chunks_of_group, h = (after_row - g * chunks_of_group) * HEADS;
                for (int i = lane; i < min(HEADS, G - h) * KS / 4; i += 32)
                    if ((i % (KS / 4)) * 64 < D)
                        prefetch_l2(a.q + after_b * a.q_request + (g * G + h + i / (KS / 4)) * a.q_head + (i % (KS / 4)) * 64);
            }
        }
        const bool full = primed == S - 1;
        if (full) cp_async_wait_group<S - 2>();
        __syncwarp();
        copy_tile(put);
        put = put + 1 == S ? 0 : put + 1;
        if (!full) {
            ++primed;
            continue;
        }
        if (t == seg.t0) {
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
                    const int eb = min(static_cast<int>(big >> 7), 254);
                    const int sh = min(141 - eb, 126);
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
        {
            const uint32_t kt = ring + slot * Sh::kStageBytes, vt = kt + kTile * Sh::kRowBytes;
            const uint32_t mask = tile_mask[warp][slot];
            slot = slot + 1 == S ? 0 : slot + 1;

            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
            if (!E4M3) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t f[4];
                    ldmatrix_x4(f, kt + tile_offset<CH>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) attn_mma<E4M3>(s[n], f[0], f[1], f[2], f[3], qf[n][k][0], qf[n][k][1]);
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
                            attn_mma<E4M3>(s[n], a0, a1, a2, a3, qf[n][k + j][0], qf[n][k + j][1]);
                    }
                }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] *= sl[n][e & 1];
                if (mask != 0xFFFFu) {
                    const bool lo = (mask >> r) & 1u, hi = (mask >> (r + 8)) & 1u;
                    if (!lo) s[n][0] = s[n][1] = -INFINITY;
                    if (!hi) s[n][2] = s[n][3] = -INFINITY;
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
                        keep[e] = m[n][e] == top[e] ? 1.f : exp2_fast(m[n][e] - top[e]);  // -inf: 0
                        m[n][e] = top[e];
                        l[n][e] *= keep[e];
                    }
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][k][e] *= keep[e & 1];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float from = m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1] - kBias;
                    s[n][e] = exp2_fast(s[n][e] - from);
                    l[n][e & 1] += s[n][e];
                }
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
            if (!E4M3) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t f[4];
                    ldmatrix_x4_trans(f, vt + tile_offset<CH>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) attn_mma<E4M3>(o[n][k], f[0], f[1], f[2], f[3], pf[n][0], pf[n][1]);
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
                        for (int n = 0; n < NT; ++n)
                            attn_mma<E4M3>(o[n][k + j], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                    }
                }
            }
        }

        if (++t < seg.t1) continue;

        // --- the result of the segment ---------------------------------------
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 16);
            }
        const bool begins = seg.t0 == 0, ends = seg.t1 == seg.q.tiles;
        if (begins && ends) {
            const float vs = E4M3 ? a.cache.v_scale[hk] : 1.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f[e] = l[n][e] != 0.f ? vs / l[n][e] : 0.f;
                    const int h = n * 8 + 2 * c + e;
                    if (a.lse && r == 0 && h < heads)
                        a.lse[static_cast<int64_t>(seg.b) * a.q_heads + head0 + h] =
                            l[n][e] != 0.f ? (m[n][e] + (log2f(l[n][e]) - kBias)) * 0.6931471805599453f : -INFINITY;
                }
                // transposed to dims along the lanes of a head
                uint16_t* out = a.out + seg.b * a.out_request + (head0 + n * 8 + r) * a.out_head;
                const bool have = n * 8 + r < heads;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(o[n][k][2 * e] * f[0], o[n][k][2 * e + 1] * f[1]);
                        v[e] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&p));
                    }
                    if (have && k * 16 < D) {
                        if (E4M3) {  // rows of the product: even dims, then odd ones
                            *reinterpret_cast<uint2*>(out + k * 16 + 4 * c) =
                                make_uint2(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[0], v[1], 0x7632));
                        } else {
                            *reinterpret_cast<uint32_t*>(out + k * 16 + 2 * c) = v[0];
                            *reinterpret_cast<uint32_t*>(out + k * 16 + 8 + 2 * c) = v[1];
                        }
                    }
                }
            }
            if (jp.split && jp.by_row && lane == 0) jp.joins[seg.b * rows + seg.row] = make_int4(-1, 0, 0, 0);
        } else {
            const int i = warp * 2 + (begins ? 1 : 0);
            if (begins) {  // the last tiles of the share: the ring is free
                cp_async_wait_group<0>();
                __syncwarp();
            }
            float* part = part_of(i);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = n * 8 + 2 * c + e;
                    if (r == 0) {
                        part_m[i][h] = m[n][e];
                        part_l[i][h] = l[n][e];
                    }
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        if (E4M3) {
                            *reinterpret_cast<float2*>(part + part_index<E4M3, DP>(h, k * 16 + 2 * r)) =
                                make_float2(o[n][k][e], o[n][k][2 + e]);
                        } else {
                            part[part_index<E4M3, DP>(h, k * 16 + r)] = o[n][k][e];
                            part[part_index<E4M3, DP>(h, k * 16 + r + 8)] = o[n][k][2 + e];
                        }
                    }
                }
            if (lane == 0) {
                part_b[i] = seg.b;
                part_row[i] = seg.row;
                part_ends[i] = (begins ? 1 : 0) | (ends ? 2 : 0);
                part_at[i] = seg.at + kRowCost;
                part_tiles[i] = seg.q.tiles;
            }
        }
        live = next_segment(seg);
        t = seg.t0;
        fresh = true;
    }
    cp_async_wait_group<0>();
    __syncthreads();

    // --- parts of one row become one -----------------------------------------
    // thread (i, h): the factor of part i's head h, and what part i leads
    for (int x = threadIdx.x; x < kAttnWarps * 2 * HEADS; x += kAttnThreads) {
        const int i = x / HEADS, h = x - i * HEADS;
        if (part_b[i] < 0) continue;
        float top = -INFINITY, all = 0.f;
        uint32_t members = 0u;
#pragma unroll 1
        for (int j = 0; j < kAttnWarps * 2; ++j)
            if (part_b[j] == part_b[i] && part_row[j] == part_row[i]) {
                members |= 1u << j;
                top = fmaxf(top, part_m[j][h]);
            }
#pragma unroll 1
        for (int j = 0; j < kAttnWarps * 2; ++j)
            if ((members >> j) & 1u)
                if (part_l[j][h] != 0.f) all += part_l[j][h] * (part_m[j][h] == top ? 1.f : exp2_fast(part_m[j][h] - top));
        part_f[i][h] = part_l[i][h] != 0.f ? (part_m[i][h] == top ? 1.f : exp2_fast(part_m[i][h] - top)) : 0.f;
        part_top[i][h] = top;
        part_all[i][h] = all;
        if (h == 0) part_members[i] = members;
    }
    if (jp.split && !jp.by_row && threadIdx.x == 0) jp.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < kAttnWarps * 2; ++i) {
        if (part_b[i] < 0) continue;
        const uint32_t members = part_members[i];
        if (members & ((1u << i) - 1u)) continue;  // an earlier part leads
        const int b = part_b[i], row = part_row[i], final_part = 31 - __clz(members);
        const int flags = part_ends[i] | part_ends[final_part];
        const int hk_i = row / chunks_of_group, chunk = row - hk_i * chunks_of_group;
        const int head_i = hk_i * G + chunk * HEADS, n = min(HEADS, G - chunk * HEADS);
        const bool whole = flags == 3;
        const float vs = E4M3 ? a.cache.v_scale[hk_i] : 1.f;
        float* const to = jp.part + (static_cast<int64_t>(blockIdx.x) * 2 + (flags & 1)) * (HEADS * (DP + 2));
#pragma unroll 1
        for (int item = threadIdx.x; item < n * (DP / 4); item += kAttnThreads) {
            const int h = item / (DP / 4), d = (item % (DP / 4)) * 4;
            if (d >= D) continue;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (uint32_t left = members; left; left &= left - 1u) {
                const int j = __ffs(left) - 1;
                const float f = part_f[j][h];
                if (f == 0.f) continue;  // nothing there: the part may hold anything
                const float4 x = *reinterpret_cast<const float4*>(part_of(j) + part_index<E4M3, DP>(h, d));
                v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y);
                v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
            }
            const float all = part_all[i][h];
            if (whole) {
                const float f = all != 0.f ? vs / all : 0.f;
                const uint32_t lo = f32_to_bf16_rn(v.x * f) | (static_cast<uint32_t>(f32_to_bf16_rn(v.y * f)) << 16);
                const uint32_t hi = f32_to_bf16_rn(v.z * f) | (static_cast<uint32_t>(f32_to_bf16_rn(v.w * f)) << 16);
                *reinterpret_cast<uint2*>(a.out + b * a.out_request + (head_i + h) * a.out_head + d) = make_uint2(lo, hi);
                if (d == 0 && a.lse)
                    a.lse[static_cast<int64_t>(b) * a.q_heads + head_i + h] =
                        all != 0.f ? (part_top[i][h] + (log2f(all) - kBias)) * 0.6931471805599453f : -INFINITY;
            } else {
                *reinterpret_cast<float4*>(to + h * DP + d) = v;
                if (d == 0) {
                    to[HEADS * DP + h] = part_top[i][h];
                    to[HEADS * (DP + 1) + h] = all;
                }
            }
        }
        // a row that begins here: what the join launch has to do for it
        if (jp.split && threadIdx.x == 0 && (flags & 1) && (jp.by_row || !whole))
            jp.joins[jp.by_row ? b * rows + row : static_cast<int>(blockIdx.x)] =
                make_int4(whole ? -1 : b, row, static_cast<int>(blockIdx.x), cta_of(part_at[i] + part_tiles[i] - 1));
    }
    if (bad) raise_device_error(a.err, W4A16_DEVERR_SLOT);
}

template <bool E4M3, int DP, int NT>
cudaError_t launch_attention_shape(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan& ws,
                                   cudaStream_t s) {
    using Sh = AttnShape<E4M3, DP, NT>;
    const void* kernel = reinterpret_cast<const void*>(k_paged_attention_mma<E4M3, DP, NT>);
    cudaError_t e = ensure_dynamic_smem(kernel, Sh::kSmem);
    if (e != cudaSuccess) return e;
    int ctas = dev.sms * Sh::kPerSm;
    if (ctas > kMostAttnCtas) ctas = kMostAttnCtas;
    ws.heads = Sh::kHeads;
    ws.padded = DP;
    ws.rows = a.cache.heads * ((a.q_heads / a.cache.heads + Sh::kHeads - 1) / Sh::kHeads);
    ws.by_row = static_cast<int64_t>(a.B) * ws.rows <= ctas;
    ws.ctas = ctas;
    // rows of few tiles: not worth a second launch, so CTAs take them whole
    ws.split = a.most > kWholeTiles * kTile;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_paged_attention_mma<E4M3, DP, NT>, a, ws);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool E4M3>
cudaError_t launch_attention_type(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan& ws,
                                  cudaStream_t s) {
    const bool wide = a.q_heads / a.cache.heads > 8;
    switch ((a.cache.dim + 63) / 64) {
        case 1: return wide ? launch_attention_shape<E4M3, 64, 2>(a, dev, ws, s) : launch_attention_shape<E4M3, 64, 1>(a, dev, ws, s);
        case 2: return wide ? launch_attention_shape<E4M3, 128, 2>(a, dev, ws, s) : launch_attention_shape<E4M3, 128, 1>(a, dev, ws, s);
        case 3: return wide ? launch_attention_shape<E4M3, 192, 2>(a, dev, ws, s) : launch_attention_shape<E4M3, 192, 1>(a, dev, ws, s);
        default: return wide ? launch_attention_shape<E4M3, 256, 2>(a, dev, ws, s) : launch_attention_shape<E4M3, 256, 1>(a, dev, ws, s);
    }
}

}  // namespace
}  // namespace w4a16
