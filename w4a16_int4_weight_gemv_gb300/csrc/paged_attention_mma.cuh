// Attention over a paged key/value cache, of one new token per request over bf16 or
// e4m3 with a scale a head (w4a16_paged_attention), of one to sixteen over 8 bits with a
// scale for each group of tokens and head (w4a16_scaled_attention): the kernels, for one
// cache type per translation unit.
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
// (tcgen05 could take 128 tokens as its rows and the heads as its columns; it was not tried.)
//
// Measured on one GB300 (copies run at 6.67 TB/s) in a CUDA graph, 32 query
// heads over 8 of 128 dims: one request of 131072 tokens in bf16 92 us (5.85
// TB/s), 128 requests of 0 to 8192 tokens over e4m3 124 us (5.88 TB/s; 58 % of
// the issue slots, 18 % of the tensor pipe), 16 requests of 0 to 4096 tokens
// 26 us (15 us of it at the rate of HBM, the rest the two launches), one request
// of 300 tokens 5.0 us.
// Registers: all instances but those of 16 heads of 256 dims (16 bytes spilled by
// the shares over bf16, 96 over e4m3, 102 in one launch) and 16 of 192 over e4m3 (32,
// in one launch 12) hold what they need.
//
// Scales by group.  A row's columns are (new token, query head) pairs.  With codes c and
// scales a (keys) and b (values),
//     s_j = c a_j q . k_j,  m = max s_j,  l = sum 2^(s_j - m),
//     w_j = s_j + log2 b_j,  M = max w_j,  o = sum 2^(w_j - M) v_j,  out = o 2^(M - m) / l:
// the value's scale goes into the weight, which is what the second product needs in fp16
// anyway, and o by a maximum of its own, since scales of neighbouring groups may be any
// powers of two apart.  m and M move only when a score passes them by 2^kSlack.
//   - A tile (32 tokens up to 128 dims) is boxes of 8, 16 or 32 tokens of a block and head,
//     each a tensor copy to the warp's ring, which its mbarrier counts: with cp.async the
//     copies were a third of all instructions.  A box's scale comes with its block id, those
//     of groups of 1, 2 or 4 tokens as small copies of their own; what fits neither comes by
//     cp.async.
//   - A CTA whose warps all lie inside of one row joins their parts itself (131072 tokens of
//     one request, heads apart: 58 us without, 53 with).
//   - Up to 32 columns take one row: the codes' conversion and the copies, of which there are
//     as many for one column as for 32, are what a tile costs.
// Bound, on a GB300 whose copies run at 6.77 TB/s (32 heads over 8 of 128 dims, int8):
//   - with one new token by HBM while there is enough to read: 64 requests of 8192 tokens 175 to
//     178 us, 6.1 TB/s; 128 of 0 to 8192 127 us, 5.7 TB/s; 32 of 8192 97 us, over the whole of
//     which DRAM is 70 % busy, issue 57 %, the ALU pipe 55 %, the tensor pipe 15 %;
//   - from 16 columns on by what eight warps an SM, all that registers hold, do one after another
//     (issue 40 to 45 %, tensor pipe 21 to 28 %): 16 requests of 8192 tokens, 268 MB, 56 us with
//     4 columns, 72 with 16, 91 with 20, 123 with 32, over e4m3 56, 64, 83 and 113;
//   - below 50 MB by two launches and their dependent reads (16 requests of 0 to 4096 tokens, a
//     scale a token, 22 us, 7.5 of it at the rate of HBM), or by one (300 tokens 6.7 us in a graph).
// Registers: the shares spill (over int8, over e4m3) 386 and 326 bytes in 16 columns of 256
// dims, 90 and 26 in 32 of 128, 8 and none in 32 of 96 and in 16 of 64, single launches 158 and
// 90, 14 and 4 in the first two; no others.
#pragma once

#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "paged_attention.h"
#include "scaled.h"

namespace w4a16 {
namespace {

// What a kernel is built for: the cache's type, and where its scales are.
constexpr int kBf16 = 0;        // none
constexpr int kE4m3 = 1;        // one a head
constexpr int kE4m3Groups = 2;  // one a group of tokens and head, as for
constexpr int kInt8Groups = 3;
constexpr bool in_8_bits(int C) { return C != kBf16; }
constexpr bool by_group(int C) { return C >= kE4m3Groups; }
template <int C>
struct ArgsOf {
    using type = AttentionArgs;
};
template <>
struct ArgsOf<kE4m3Groups> {
    using type = ScaledAttentionArgs;
};
template <>
struct ArgsOf<kInt8Groups> {
    using type = ScaledAttentionArgs;
};
template <int C>
using Args = typename ArgsOf<C>::type;

// Scales by group: weights go into fp16 products as 2^kWeightBias of the largest,
// which may grow by 2^kSlack before o is scaled again: 2^15 at most.
constexpr float kWeightBias = 8.f, kSlack = 7.f;

// Tokens of a tile: the MMA's rows; with scales by group twice as many, whose control then
// weighs half as much a token, where a ring of those fits.
constexpr int tile_tokens(int C, int DP) { return by_group(C) && DP <= 128 ? 32 : kTile; }

constexpr int kMinCost = 3;     // a warp's share at least
constexpr int kTeamTiles = 5;   // and where it takes the same tokens of its request's heads as its neighbours
constexpr int kTeamRow = 1 << 30;  // a row (below 2^24) to join of which each warp has a part
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
// A word of four codes as two fp16 pairs, exactly: e4m3 the first two and the last
// two, int8 the first and third and the second and fourth.
template <int C>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (C == kInt8Groups) {
        // 1024 + (code + 128), the code's byte (its top bit turned) as the low one of an fp16
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        const uint32_t x = (w & 0x00FF00FFu) ^ 0x64806480u, y = ((w >> 8) & 0x00FF00FFu) ^ 0x64806480u;
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&x), off), b = __hsub2(*reinterpret_cast<const __half2*>(&y), off);
        lo = *reinterpret_cast<const uint32_t*>(&a), hi = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        lo = e4m3x2_to_f16x2(w), hi = e4m3x2_to_f16x2(w >> 16);
    }
}
// A word of four codes, two dims (even, odd) of one token, then of the next, as the fp16
// pairs of the even and of the odd dim.
template <int C>
__device__ __forceinline__ void codes_to_f16_by_dim(uint32_t w, uint32_t& even, uint32_t& odd) {
    codes_to_f16<C>(C == kInt8Groups ? w : __byte_perm(w, 0u, 0x3120), even, odd);
}
__device__ __forceinline__ void cp_async_4_zfill(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_u4(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// log2 of a scale's magnitude
__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(fabsf(x)));
    return y;
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
template <int C>
__device__ __forceinline__ void attn_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (in_8_bits(C)) {
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

// The same where scales go by group: as a tensor copy lays boxes of 64 or 128 bytes by
// tokens out, of 256-byte rows the first halves of all tokens and then the second.
template <int CH>
__device__ __forceinline__ uint32_t group_offset(int r, int c) {
    if (CH == 4) return static_cast<uint32_t>((r * 4 + (c ^ ((r >> 1) & 3))) * 16);
    return static_cast<uint32_t>((c >> 3) * (kTile * 128) + (r * 8 + ((c & 7) ^ (r & 7))) * 16);  // (two halves: tiles of kTile)
}

template <int C, int DP, int NT>
struct AttnShape {
    static constexpr int kHeads = 8 * NT;
    static constexpr int kSteps = DP / 16;                     // 16-dim steps of a head
    // 16-byte chunks of a row in shared memory (six would not swizzle: eight)
    // (scales by group: as the tensor copies lay rows out, 64 bytes or one or two times 128)
    static constexpr bool k8 = in_8_bits(C);
    static constexpr int kChunks = by_group(C) ? (DP == 64 ? 4 : DP <= 128 ? 8 : 16) : k8 && DP == 96 ? 8 : DP * (k8 ? 1 : 2) / 16;
    static constexpr int kRowBytes = kChunks * 16;
    static constexpr int kTokens = tile_tokens(C, DP);
    static constexpr int kStageBytes = 2 * kTokens * kRowBytes;  // keys, then values
    // Scales by group: what is known of a tile in shared memory.  For every eight of its tokens 16
    // bytes: the mask of those that the row sees, their keys' and their values' scale
    // (kBoxScales); then the scales of its tokens' keys and of their values, one by one.
    static constexpr int kInfoKeys = kTokens * 2, kInfoValues = kTokens * 6, kInfo = kTokens * 10;
    // that and a barrier are beside a stage; and what aligns the first one
    static constexpr int kBeside = by_group(C) ? kInfo + 8 : 0, kAlign = by_group(C) ? 1024 : 0;
    // more than 16 heads: their queries, which registers do not hold beside the sums, of each warp
    static constexpr int kQueries = NT > 2 ? NT * kSteps * 256 : 0;
    static constexpr int kPartFloats = kHeads * (DP + 2);
    // shares: one CTA an SM, of as many warps as its registers allow (the accumulators'
    // size decides) with rings of three stages or more
    static constexpr int kShareWarps = 4 * (k8 ? (NT == 1 ? (DP == 64 ? 4 : DP <= 128 ? 3 : 2) : (DP == 64 && NT == 2 ? 3 : 2))
                                                 : (DP == 64 ? 3 : DP <= 128 ? 2 : 1));
    static constexpr int kFit = (226 * 1024 - kAlign - kShareWarps * kQueries) / (kShareWarps * (kStageBytes + kBeside));
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kSmem = kShareWarps * (kStages * (kStageBytes + kBeside) + kQueries) + kAlign;
    // rows: one CTA an SM
    static constexpr int kRowWarps = kStageBytes > 12288 ? 4 : 8;
    static constexpr int kRowFit = (225 * 1024 - kAlign - kRowWarps * kQueries) / (kRowWarps * (kStageBytes + kBeside));
    static constexpr int kRowStages = kRowFit > 4 ? 4 : kRowFit;
    static constexpr int kRowRing = kRowStages * kStageBytes;  // of a warp
    static constexpr int kRowSmem = kRowWarps * (kRowRing + kRowStages * kBeside + kQueries) + kAlign;
    // scales by group: how many 16 tokens are worked on together.  Two for up to 24 columns
    // (drafts of 4 tokens of 4 heads, 16 x 8192 tokens of int8 77 -> 70 us; of 5 tokens 96 ->
    // 91), one for 32, whose registers then spill twice as much (121 -> 131).
    static constexpr int kTogether = kTokens == 32 && NT <= 3 ? 2 : 1;
    static constexpr int kPartBytes = kHeads * DP * 4;
    static constexpr bool kClusters = kRowRing >= 2 * kPartBytes;  // room for the CTA's part behind a warp's
    static_assert(kStages >= (kTokens == 32 ? 2 : 3), "ring too short");
    static_assert(kRowStages >= 2 && kRowRing >= kPartBytes, "no room for a warp's part");
    static_assert(160 * kShareWarps <= most_workers(DP), "workspace");
    static_assert(!by_group(C) || kStages * kStageBytes >= kPartBytes, "no room for a warp's part");
};

// New tokens of a request.
template <int C>
__device__ __forceinline__ int new_tokens(const Args<C>& a) {
    if constexpr (by_group(C)) return a.tokens;
    else return 1;
}

// Whether tiles come as groups of cp.async.
template <int C>
__device__ __forceinline__ bool counts_groups(const Args<C>& a) {
    if constexpr (by_group(C)) return a.scales == kTokenScales;
    else return true;
}

// What one request looks like: its visible tokens [start, len), in tiles from
// tile0 on (visible to any of its new tokens).
struct Request {
    int len, start, tile0, tiles;
};

template <int C, int TOKENS>
__device__ __forceinline__ Request request_of(const Args<C>& a, int b, bool& bad) {
    Request q;
    const int len = a.kv_len[b];
    bad |= len < 0 || len > a.most;
    q.len = min(max(len, 0), a.most);
    q.start = a.window > 0 ? max(q.len - (new_tokens<C>(a) - 1) - a.window, 0) : 0;
    q.tile0 = q.start / TOKENS;
    q.tiles = q.len > 0 ? (q.len - 1) / TOKENS + 1 - q.tile0 : 0;
    return q;
}

// Which heads row `row` of a request stands for.  With scales by group these are (new
// token, query head) pairs, those of the first token first.
struct Heads {
    int hk, first, n;  // key/value head, first query head (by group: first pair of those that share hk), how many
};
template <int C, int HEADS>
__device__ __forceinline__ Heads heads_of(const Args<C>& a, int row) {
    const int G = a.q_heads / a.cache.heads * new_tokens<C>(a), chunks = (G + HEADS - 1) / HEADS;
    Heads h;
    h.hk = row / chunks;
    const int chunk = row - h.hk * chunks;
    h.first = chunk * HEADS + (by_group(C) ? 0 : h.hk * G);
    h.n = min(HEADS, G - chunk * HEADS);
    return h;
}
// The new token and the query head of a row's j-th.
struct Column {
    int token, head;
};
template <int C>
__device__ __forceinline__ Column column_of(const Args<C>& a, const Heads& hd, int j) {
    Column c{0, hd.first + j};
    if constexpr (by_group(C)) {
        const int G = a.q_heads / a.cache.heads;
        c.token = c.head / G;
        c.head -= c.token * G;
        c.head += hd.hk * G;
    }
    return c;
}
template <int C>
__device__ __forceinline__ const uint16_t* query_of(const Args<C>& a, int b, const Heads& hd, int j) {
    const Column c = column_of<C>(a, hd, j);
    const uint16_t* q = a.q + b * a.q_request + c.head * a.q_head;
    if constexpr (by_group(C)) q += c.token * a.q_token;
    return q;
}
template <int C>
__device__ __forceinline__ uint16_t* out_of(const Args<C>& a, int b, const Heads& hd, int j) {
    const Column c = column_of<C>(a, hd, j);
    uint16_t* out = a.out + b * a.out_request + c.head * a.out_head;
    if constexpr (by_group(C)) out += c.token * a.out_token;
    return out;
}
template <int C>
__device__ __forceinline__ float* lse_at(const Args<C>& a, int b, const Heads& hd, int j) {
    const Column c = column_of<C>(a, hd, j);
    return a.lse + (static_cast<int64_t>(b) * new_tokens<C>(a) + c.token) * a.q_heads + c.head;
}

template <int C>
__device__ __forceinline__ void store_empty(const Args<C>& a, int b, const Heads& hd, int thread, int threads) {
    const int per = a.cache.dim / 8;
    for (int i = thread; i < hd.n * per; i += threads)
        *reinterpret_cast<uint4*>(out_of<C>(a, b, hd, i / per) + (i % per) * 8) = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
        for (int j = thread; j < hd.n; j += threads) *lse_at<C>(a, b, hd, j) = -INFINITY;
}

// 16 dims of 8 heads from the accumulators (row r and r + 8 by columns 2c,
// 2c + 1) times the heads' factors, transposed to dims along the lanes of a
// head and stored; `out`: the row of head r's output, null for none.
template <int C>
__device__ __forceinline__ void store_dims(const float4& o, float f0, float f1, uint16_t* out, int c) {
    const __nv_bfloat162 p0 = __floats2bfloat162_rn(o.x * f0, o.y * f1), p1 = __floats2bfloat162_rn(o.z * f0, o.w * f1);
    const uint32_t v0 = transpose_8x8(*reinterpret_cast<const uint32_t*>(&p0));
    const uint32_t v1 = transpose_8x8(*reinterpret_cast<const uint32_t*>(&p1));
    if (!out) return;
    if (in_8_bits(C)) {  // rows of the product: even dims, then odd ones
        *reinterpret_cast<uint2*>(out + 4 * c) = make_uint2(__byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632));
    } else {
        *reinterpret_cast<uint32_t*>(out + 2 * c) = v0;
        *reinterpret_cast<uint32_t*>(out + 8 + 2 * c) = v1;
    }
}
template <int C>
__device__ __forceinline__ float lse_of(float m, float l) {
    return l != 0.f ? (m + (log2f(l) - (C == kE4m3 ? kE4m3Bias : 0.f))) * 0.6931471805599453f : -INFINITY;
}

// The arithmetic of a warp on tiles of one row.  Lane 4 r + c.
template <int C, int DP, int NT>
struct RowMath {
    using Sh = AttnShape<C, DP, NT>;
    static constexpr int CH = Sh::kChunks, KS = Sh::kSteps;
    static constexpr bool kQueriesNear = NT > 2;  // in shared memory: [step][head block][lane] pairs of words
    uint32_t qf[kQueriesNear ? 1 : NT][KS][2];    // queries as B fragments (columns: heads)
    uint32_t queries;                             // or where those are
    float sl[NT][2];                     // score scale of columns 2c, 2c + 1
    float m[NT][2], l[NT][2];            // of columns 2c, 2c + 1 (l: of this lane's tokens until reduced)
    float4 o[NT][KS];                    // dims r, r + 8 (8 bits: 2r, 2r + 1) by columns 2c, 2c + 1
    // with scales by group, where a value's weight is p times its scale: the largest weight
    // (log2 units), by which o is scaled, and the tokens that the column sees, below
    // upto, of them the last `window`
    float big[NT][2];
    int upto[NT][2];

    // the queries of head block n
    __device__ __forceinline__ void request(const Args<C>& a, int b, const Heads& hd, int n, uint32_t (&q)[KS][2], int lane) const {
        const int r = lane >> 2, c = lane & 3;
        const uint16_t* qp = query_of<C>(a, b, hd, n * 8 + r);
        const bool have = n * 8 + r < hd.n;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            q[k][0] = q[k][1] = 0u;
            if (have && k * 16 < a.cache.dim) {
                // bf16: dims 2c, 2c + 1 and 8 further; 8 bits: the four dims whose codes one word holds
                const int d = k * 16 + (in_8_bits(C) ? 4 * c : 2 * c);
                q[k][0] = *reinterpret_cast<const uint32_t*>(qp + d);
                q[k][1] = *reinterpret_cast<const uint32_t*>(qp + d + (in_8_bits(C) ? 2 : 8));
            }
        }
    }

    // requests the queries and clears the sums
    __device__ __forceinline__ void begin(const Args<C>& a, int b, const Heads& hd, int lane) {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (!kQueriesNear) request(a, b, hd, n, qf[kQueriesNear ? 0 : n], lane);
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
                if constexpr (by_group(C)) {
                    big[n][e] = -INFINITY;
                    upto[n][e] = column_of<C>(a, hd, n * 8 + 2 * c + e).token + 1 - a.tokens;  // and its length: ready()
                }
            }
        }
    }

    // makes the queries that begin() requested into operands
    __device__ __forceinline__ void ready(const Args<C>& a, int b, const Heads& hd, int len, int lane) {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            sl[n][0] = sl[n][1] = a.scale * 1.4426950408889634f * (C == kE4m3 ? a.cache.k_scale[hd.hk] : 1.f);
            if (by_group(C)) upto[n][0] += len, upto[n][1] += len;
            if (in_8_bits(C)) {
                if (kQueriesNear) request(a, b, hd, n, qf[0], lane);
                uint32_t(&q)[KS][2] = qf[kQueriesNear ? 0 : n];
                // to fp16, scaled by a power of two that takes the head's largest into [2^14, 2^15)
                uint32_t big = 0u;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    big = __vmaxu2(big, __vmaxu2(q[k][0] & 0x7FFF7FFFu, q[k][1] & 0x7FFF7FFFu));
                big = max(big & 0xFFFFu, big >> 16);
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                const int sh = min(141 - min(static_cast<int>(big >> 7), 254), 126);
                const float up = exp2i(sh), down = exp2i(-sh);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t v = q[k][e];
                        const __half2 h = __floats2half2_rn(bf16_to_f32(v & 0xFFFFu) * up, bf16_to_f32(v >> 16) * up);
                        q[k][e] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    if (C == kInt8Groups) {  // the pairs that codes_to_f16 makes
                        const uint32_t v0 = q[k][0], v1 = q[k][1];
                        q[k][0] = __byte_perm(v0, v1, 0x5410), q[k][1] = __byte_perm(v0, v1, 0x7632);
                    }
                    if (kQueriesNear)
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(queries + ((k * NT + n) * 32 + lane) * 8), "r"(q[k][0]), "r"(q[k][1]) : "memory");
                }
                sl[n][0] *= __shfl_sync(0xFFFFFFFFu, down, 8 * c);
                sl[n][1] *= __shfl_sync(0xFFFFFFFFu, down, 8 * c + 4);
            }
        }
    }

    // the largest of a column's tokens
    static __device__ __forceinline__ float over_tokens(float x) {
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
        return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
    }
    __device__ __forceinline__ void scale_o(int n, const float (&f)[2]) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            o[n][k].x *= f[0], o[n][k].y *= f[1];
            o[n][k].z *= f[0], o[n][k].w *= f[1];
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
        if (!in_8_bits(C)) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t f[4];
                ldmatrix_x4(f, kt + tile_offset<CH>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
                for (int n = 0; n < NT; ++n) attn_mma<C>(kTwo && (k & 1) ? s1[n] : s[n], f[0], f[1], f[2], f[3], qf[n][k][0], qf[n][k][1]);
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
                        attn_mma<C>(kTwo && j ? s1[n] : s[n], a0, a1, a2, a3, qf[n][k + j][0], qf[n][k + j][1]);
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
            for (int e = 0; e < 2; ++e) top[e] = fmaxf(over_tokens(top[e]), m[n][e]);
            if (__any_sync(0xFFFFFFFFu, top[0] > m[n][0] || top[1] > m[n][1])) {
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    keep[e] = part_factor(m[n][e], top[e]);  // from -infinity: 0
                    m[n][e] = top[e];
                    l[n][e] *= keep[e];
                }
                scale_o(n, keep);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // the bias after the difference: m - 15 is not a float where m passes 2^24, and
                // the largest p would then be 2^16, which no fp16 holds
                s[n][e] -= m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1];
                s[n][e] = exp2_fast(C == kE4m3 ? s[n][e] + kE4m3Bias : s[n][e]);
                l[n][e & 1] += s[n][e];
            }
            // to 16 bits for the second product, whose operands are of one type: that of the
            // values.  fp16 rounds p by 2^-11 of it, bf16 by 2^-8, about as much as the result's
            // own rounding; l takes the unrounded ones.  (131072 tokens in bf16: 0.0020 off in
            // all, 0.0017 with fp32 weights; over e4m3 no difference shows.)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t v;
                if (in_8_bits(C)) {
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
            attn_mma<C>(d, a0, a1, a2, a3, pf[n][0], pf[n][1]);
            o[n][k] = make_float4(d[0], d[1], d[2], d[3]);
        };
        if (!in_8_bits(C)) {
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

    // --- scales by group ------------------------------------------------------
    // Scores s of P tiles (log2 units; rows r, r + 8 by columns 2c, 2c + 1) to the weights of
    // the values, p times the scale, 2^lv.  o goes by the largest weight: by the largest p instead,
    // a token of large scale and small p would pass what fp16 holds.  m and the largest weight
    // need not be the largest there are, only near them (kSlack), so that most tiles take a vote
    // here and no exchange.  HIDDEN: some scores are -infinity for tokens that a column does not
    // see, whose scale may be anything.
    template <int P, bool HIDDEN>
    __device__ __forceinline__ void weigh(int n, float (&s)[P][NT][4], const float (&lv)[P][2], const uint32_t (&sign)[P][2]) {
        float top[2], heavy[2];
        const auto weight = [&](int p, int e) { return HIDDEN && s[p][n][e] == -INFINITY ? -INFINITY : s[p][n][e] + lv[p][e >> 1]; };
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[e] = heavy[e] = -INFINITY;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                top[e] = fmaxf(top[e], fmaxf(s[p][n][e], s[p][n][e + 2]));
                heavy[e] = fmaxf(heavy[e], fmaxf(weight(p, e), weight(p, e + 2)));
            }
        }
        bool over = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) over |= top[e] > m[n][e] + kSlack || heavy[e] > big[n][e] + kSlack;
        if (__any_sync(0xFFFFFFFFu, over)) {
            float keep[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(over_tokens(top[e]), m[n][e]);
                heavy[e] = fmaxf(over_tokens(heavy[e]), big[n][e]);
                l[n][e] *= part_factor(m[n][e], top[e]);  // from -infinity: 0
                keep[e] = part_factor(big[n][e], heavy[e]);
                m[n][e] = top[e], big[n][e] = heavy[e];
            }
            scale_o(n, keep);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float base = m[n][e] == -INFINITY ? 0.f : m[n][e], heavy = big[n][e] == -INFINITY ? 0.f : big[n][e];
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float& x = s[p][n][2 * i + e];
                    // (the bias after the difference, which is a float's whatever the maximum's size)
                    const float w = weight(p, 2 * i + e) - heavy + kWeightBias;
                    l[n][e] += exp2_fast(x - base);
                    x = __uint_as_float(__float_as_uint(exp2_fast(w)) ^ sign[p][i]);
                }
        }
    }

    // P times 16 tokens of a tile from its `from`-th on: codes at kt (shared address: keys, then
    // values), what is known of them at info; first: the number of its first token
    template <int P>
    __device__ __forceinline__ void tokens(const Args<C>& a, const Request& q, uint32_t kt, uint32_t info, int first, int from, int lane) {
        constexpr int kValues = Sh::kTokens * Sh::kRowBytes;  // from a key's place to its value's
        constexpr bool kTwo = P == 1 && NT * KS <= 16;  // two chains of products, as above
        const int r = lane >> 2;
        uint32_t at[P];  // chunk lane / 16 of row lane % 16; chunk k + lane / 16 (k even): its address xor 16 k
#pragma unroll
        for (int p = 0; p < P; ++p) at[p] = kt + (from + 16 * p) * Sh::kRowBytes + group_offset<CH>(lane & 15, lane >> 4);
        first += from;
        float s[P][NT][4], s1[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s1[n][e] = 0.f;
#pragma unroll
                for (int p = 0; p < P; ++p) s[p][n][e] = 0.f;
            }
#pragma unroll
        for (int k = 0; k < KS; k += 2)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                uint32_t f[4];  // two chunks of 16 codes: rows r and r + 8 of each
                ldmatrix_x4(f, (at[p] ^ ((k & 7) * 16)) + (k >> 3) * (kTile * 128));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t a0, a1, a2, a3;
                    codes_to_f16<C>(f[2 * j], a0, a2);
                    codes_to_f16<C>(f[2 * j + 1], a1, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t q0, q1;
                        if constexpr (kQueriesNear) {
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(q0), "=r"(q1) : "r"(queries + (((k + j) * NT + n) * 32 + lane) * 8) : "memory");
                        } else {
                            q0 = qf[n][k + j][0], q1 = qf[n][k + j][1];
                        }
                        attn_mma<C>(kTwo && j ? s1[n] : s[p][n], a0, a1, a2, a3, q0, q1);
                    }
                }
            }
        uint32_t mask[P], pf[P][NT][2];
        float ks[P][2], lv[P][2];
        uint32_t sign[P][2];
        bool hidden = false;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint32_t known = info + (from + 16 * p) * 2;
            const uint4 x = ld_shared_u4(known), y = ld_shared_u4(known + 16);  // rows r, rows r + 8
            mask[p] = x.x | (y.x << 8);
            hidden |= mask[p] != 0xFFFFu;
            float v[2] = {__uint_as_float(x.z), __uint_as_float(y.z)};
            ks[p][0] = __uint_as_float(x.y), ks[p][1] = __uint_as_float(y.y);
            if (a.scales != kBoxScales) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t of = info + ((from + 16 * p + r + 8 * i) >> a.group_log2) * 4;
                    ks[p][i] = ld_shared_f32(of + Sh::kInfoKeys);
                    v[i] = ld_shared_f32(of + Sh::kInfoValues);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                lv[p][i] = log2_fast(v[i]);
                sign[p][i] = __float_as_uint(v[i]) & 0x80000000u;
            }
        }
        // tokens that some new ones see and others do not
        const bool edge = first + 16 * P > q.len - (a.tokens - 1) || (a.window > 0 && first < q.len - a.window);
        hidden |= edge;
        const auto scores = [&](int n) {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[p][n][e] = (kTwo ? s[p][n][e] + s1[n][e] : s[p][n][e]) * (sl[n][e & 1] * ks[p][e >> 1]);
        };
        const auto to_f16 = [&](int n) {  // for the second product: 2^-11 of each weight, l takes the unrounded p
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const __half2 h = __floats2half2_rn(s[p][n][2 * e], s[p][n][2 * e + 1]);
                    pf[p][n][e] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h));
                }
        };
        if (!hidden) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                scores(n);
                weigh<P, false>(n, s, lv, sign);
                to_f16(n);
            }
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (C == kE4m3Groups) {
                    // A weight of 0 does not stop a NaN: codes that no new token sees, which may be
                    // anything, become 0 where they are.  So do NaN codes that some see and others do
                    // not; the token's weight becomes NaN instead, for those that do.  (As numbers in
                    // the products' loop instead, which has no room for it: 32 columns of 128 dims 118
                    // us, so 113, 16 of 256 198, so 148; eight requests of 301 tokens 6.8, so 7.0.)
                    const int row = lane & 15, token = first + 16 * p + row;
                    const bool none = !((mask[p] >> row) & 1u);
                    const bool some = !none && edge && a.tokens > 1 && (token >= q.len - (a.tokens - 1) || (a.window > 0 && token < q.len - a.window));
                    bool nan = false;
                    if (none || some) {
#pragma unroll 1
                        for (int k = 0; k < KS; k += 2) {  // (the chunks that the products take: of 96 dims not all)
                            const uint32_t chunk = (at[p] ^ ((k & 7) * 16)) + (k >> 3) * (kTile * 128) + kValues;
                            const uint4 v = none ? make_uint4(0u, 0u, 0u, 0u) : ld_shared_u4(chunk);
                            uint32_t x[4] = {v.x, v.y, v.z, v.w}, found = 0u;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t top = ((x[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // of bytes 0x7F, 0xFF
                                found |= top;
                                x[j] &= ~((top >> 7) * 0xFFu);
                            }
                            nan |= found != 0u;
                            if (none || found) st_shared_u4(chunk, make_uint4(x[0], x[1], x[2], x[3]));
                        }
                    }
                    fence_proxy_async_smem();  // before the next tensor copy into this stage
                    uint32_t who = __ballot_sync(0xFFFFFFFFu, nan);
                    who |= who >> 16;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if ((who >> (r + 8 * i)) & 1u) lv[p][i] = NAN;
                    __syncwarp();
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                scores(n);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (!((mask[p] >> r) & 1u)) s[p][n][0] = s[p][n][1] = -INFINITY;
                    if (!((mask[p] >> (r + 8)) & 1u)) s[p][n][2] = s[p][n][3] = -INFINITY;
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int token = first + 16 * p + r + 8 * (e >> 1), end = upto[n][e & 1];
                            if (token >= end || (a.window > 0 && token < end - a.window)) s[p][n][e] = -INFINITY;
                        }
                    }
                }
                weigh<P, true>(n, s, lv, sign);
                to_f16(n);
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                uint32_t f[4];  // chunk k: tokens 0..7, 8..15, then chunk k + 1
                ldmatrix_x4_trans(f, (at[p] ^ ((k & 7) * 16)) + (k >> 3) * (kTile * 128) + kValues);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // word: dims 2r, 2r + 1 of token 2c, then of token 2c + 1
                    uint32_t a0, a1, a2, a3;
                    codes_to_f16_by_dim<C>(f[2 * j], a0, a1);
                    codes_to_f16_by_dim<C>(f[2 * j + 1], a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float d[4] = {o[n][k + j].x, o[n][k + j].y, o[n][k + j].z, o[n][k + j].w};
                        attn_mma<C>(d, a0, a1, a2, a3, pf[p][n][0], pf[p][n][1]);
                        o[n][k + j] = make_float4(d[0], d[1], d[2], d[3]);
                    }
                }
            }
    }

    // a tile
    __device__ __forceinline__ void tile(const Args<C>& a, const Request& q, uint32_t kt, uint32_t info, int first, int lane) {
        constexpr int P = Sh::kTogether;
#pragma unroll 1
        for (int from = 0; from < Sh::kTokens; from += 16 * P) tokens<P>(a, q, kt, info, first, from, lane);
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
        if constexpr (by_group(C)) {
            // o by the largest p like l, in two steps: a float's range may not hold the factor
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    f[e] = big[n][e] == -INFINITY ? 0.f : exp2_fast(0.5f * (big[n][e] - kWeightBias - m[n][e]));
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    o[n][k].x = o[n][k].x * f[0] * f[0], o[n][k].y = o[n][k].y * f[1] * f[1];
                    o[n][k].z = o[n][k].z * f[0] * f[0], o[n][k].w = o[n][k].w * f[1] * f[1];
                }
            }
        }
    }

    // the row's result, all of its tokens seen (after reduce())
    __device__ __forceinline__ void finish(const Args<C>& a, int b, const Heads& hd, int lane) {
        const int r = lane >> 2, c = lane & 3;
        const float vs = C == kE4m3 ? a.cache.v_scale[hd.hk] : 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[e] = l[n][e] != 0.f ? vs / l[n][e] : 0.f;
                const int h = n * 8 + 2 * c + e;
                if (a.lse && r == 0 && h < hd.n) *lse_at<C>(a, b, hd, h) = lse_of<C>(m[n][e], l[n][e]);
            }
            uint16_t* out = out_of<C>(a, b, hd, n * 8 + r);
            const bool have = n * 8 + r < hd.n;
#pragma unroll
            for (int k = 0; k < KS; ++k)
                store_dims<C>(o[n][k], f[0], f[1], have && k * 16 < a.cache.dim ? out + k * 16 : nullptr, c);
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
template <int C, int DP, int NT>
struct TileCopy {
    using Sh = AttnShape<C, DP, NT>;
    static constexpr int CH = Sh::kChunks, kBytes = in_8_bits(C) ? 1 : 2;
    int base, id, place;

    static __device__ __forceinline__ bool aligned(const Args<C>& a) { return a.cache.page % kTile == 0; }

    // the ids for tile t (tiles of the row step apart, below t1)
    __device__ __forceinline__ void look_up(const Args<C>& a, int b, const Request& q, int t, int t1, int step, int lane) {
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
    __device__ __forceinline__ bool wants(const Args<C>& a, int t, int step) const {
        return aligned(a) ? t - base >= 32 * step : t != base;
    }

    // starts the copies of tile t into dst; returns the mask of the tokens the row sees
    __device__ __forceinline__ uint32_t copy(const Args<C>& a, int hk, const Request& q, int t, int step, uint32_t dst, int lane,
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

// A tensor copy of a box (64 or 128 bytes of one head by box tokens of a block).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Scales by group: the ring of a warp, and what fills it.  Block ids are loaded early, those
// of 32 boxes at once (lane i: box i % boxes of the i / boxes-th tile).  The lane that has a
// box's id starts its copies: of the codes as tensor copies, which take next to no
// instructions (with cp.async these were a third of all); its scale comes with the id
// (kBoxScales), or those of its tokens as another copy (kRowScales).  Blocks and scales that
// do not allow that: by cp.async (kTokenScales), their codes too where no box divides a page.
template <int C, int DP, int NT>
struct GroupRing {
    using Sh = AttnShape<C, DP, NT>;
    static constexpr int CH = Sh::kChunks, kInner = CH == 4 ? 64 : 128, kHalves = CH == 16 ? 2 : 1, TT = Sh::kTokens;
    uint32_t codes, info, bars;  // shared addresses: of stage 0 its codes; what is known of it; its barrier
    int known, id, place;        // how many tiles' ids are left; this lane's
    float ks, vs;
    bool late, drained;          // a copy did not arrive; the others were waited for

    __device__ __forceinline__ void open(const Args<C>& a, uint32_t smem, int warp, int warps, int stages, int lane) {
        smem = (smem + 1023u) & ~1023u;
        codes = smem + warp * stages * Sh::kStageBytes;
        info = smem + warps * stages * Sh::kStageBytes + warp * stages * Sh::kInfo;
        bars = smem + warps * stages * (Sh::kStageBytes + Sh::kInfo) + warp * stages * 8;
        late = drained = false;
        if (lane < stages)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + lane * 8), "r"(a.scales == kTokenScales ? 1 : boxes(a)) : "memory");
        mbar_init_fence();
        fence_proxy_async_smem();
        __syncwarp();
    }
    static __device__ __forceinline__ int boxes_log2(const Args<C>& a) { return (TT == 32 ? 5 : 4) - a.box_log2; }
    static __device__ __forceinline__ int boxes(const Args<C>& a) { return TT >> a.box_log2; }

    // the ids of the boxes from tile t on (tiles step apart, below t1) that hold tokens of [low, high)
    __device__ __forceinline__ void look_up(const Args<C>& a, int b, int hk, int tile0, int low, int high, int t, int t1, int step, int lane) {
        const int shift = boxes_log2(a), tile = t + (lane >> shift) * step;
        const int token = (tile0 + tile) * TT + ((lane & (boxes(a) - 1)) << a.box_log2);
        const int col = static_cast<int>(static_cast<unsigned>(token) / static_cast<unsigned>(a.cache.page));
        place = token - col * a.cache.page;
        id = -1;
        known = 32 >> shift;
        if (tile < t1 && token < high && token + (1 << a.box_log2) > low) id = a.block_table[b * a.table_stride + col];
        if (a.scales == kBoxScales) {
            ks = vs = 0.f;
            if (id >= 0 && id < a.cache.blocks) {
                const int64_t of = __umulhi(place, a.magic);  // (a group of 8 tokens at least)
                ks = a.k_scale[id * a.ks_block + of * a.ks_group + hk * a.ks_head];
                vs = a.v_scale[id * a.vs_block + of * a.vs_group + hk * a.vs_head];
            }
        }
    }

    // kBoxScales, kRowScales: starts the copies of the row's t-th tile, the next of those looked
    // up, into a stage
    __device__ __forceinline__ void copy_boxes(const Args<C>& a, int hk, const Request& q, int t, int stage, int lane, bool& bad) {
        const int box = lane - 32 + (known << boxes_log2(a));
        --known;
        if (static_cast<unsigned>(box) < static_cast<unsigned>(boxes(a))) {
            const int u = 1 << a.box_log2, first = (q.tile0 + t) * TT + box * u;
            // the tokens from `start` on, below `len`
            const int begin = min(max(q.start - first, 0), u), end = min(max(q.len - first, 0), u);
            uint32_t mask = end > begin ? (0xFFFFFFFFu >> (32 - end)) & (0xFFFFFFFFu << begin) : 0u;
            if (id < 0 || id >= a.cache.blocks) {
                bad |= mask != 0u;
                mask = 0u;
            }
            const uint32_t dst = codes + stage * Sh::kStageBytes + box * u * kInner, bar = bars + stage * 8, to = info + stage * Sh::kInfo;
            const bool rows = a.scales == kRowScales;
            const uint32_t more = rows ? static_cast<uint32_t>(u >> a.group_log2) * 4u : 0u;  // bytes of the tokens' scales
            if (mask) {
                expect_bytes(bar, u * 2 * kHalves * kInner + 2 * more);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    tma_load_4d(dst + h * (kTile * 128), &a.k_map, h * 128, hk, place, id, bar);
                    tma_load_4d(dst + h * (kTile * 128) + TT * Sh::kRowBytes, &a.v_map, h * 128, hk, place, id, bar);
                }
                if (rows) {
                    const int64_t of = place >> a.group_log2;
                    bulk_load(to + Sh::kInfoKeys + box * more, a.k_scale + id * a.ks_block + of + hk * a.ks_head, more, bar);
                    bulk_load(to + Sh::kInfoValues + box * more, a.v_scale + id * a.vs_block + of + hk * a.vs_head, more, bar);
                }
            } else {
                expect_bytes(bar, 0);
            }
#pragma unroll
            for (int i = 0; i < TT / 8; ++i)
                if (i < u / 8)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %1};" ::"r"(to + (box * (u / 8) + i) * 16), "r"((mask >> (8 * i)) & 0xFFu),
                                 "r"(__float_as_uint(ks)), "r"(__float_as_uint(vs))
                                 : "memory");
        }
    }

    // kTokenScales: those of the next tile, the row's t-th, into a stage
    __device__ __forceinline__ void copy(const Args<C>& a, int hk, const Request& q, int t, int stage, int lane, bool& bad) {
        const uint32_t dst = codes + stage * Sh::kStageBytes, bar = bars + stage * 8, to = info + stage * Sh::kInfo;
        const int from = 32 - (known << boxes_log2(a)), u = 1 << a.box_log2;
        --known;
        const int mine = lane & (TT - 1), token = (q.tile0 + t) * TT + mine, box = from + (mine >> a.box_log2);
        const int block = __shfl_sync(0xFFFFFFFFu, id, box), in = __shfl_sync(0xFFFFFFFFu, place, box) + (mine & (u - 1));
        const bool seen = token >= q.start && token < q.len, valid = seen && block >= 0 && block < a.cache.blocks;
        bad |= seen && !valid;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, valid) & (0xFFFFFFFFu >> (32 - TT));
        const int64_t at = valid ? block : 0, row = valid ? in : 0;
        {
            const int64_t of = a.magic ? static_cast<int>(__umulhi(in, a.magic)) : in;
            const float* k = a.k_scale + at * a.ks_block + of * a.ks_group + hk * a.ks_head;
            const float* v = a.v_scale + at * a.vs_block + of * a.vs_group + hk * a.vs_head;
            if (lane < TT) {
                cp_async_4_zfill(to + Sh::kInfoKeys + mine * 4, valid ? k : a.k_scale, valid);
                cp_async_4_zfill(to + Sh::kInfoValues + mine * 4, valid ? v : a.v_scale, valid);
            }
        }
        if (lane < TT / 8) asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + lane * 16), "r"((mask >> (8 * lane)) & 0xFFu) : "memory");
        if (a.tensor_copies) {
            // lane i: of box i / (2 kHalves) the key's or the value's, first or second half
            const uint32_t here = 0xFFFFFFFFu >> (32 - u);
            const int mybox = lane / (2 * kHalves), h = lane / 2 % kHalves;
            const bool mybox_seen = mybox < boxes(a) && ((mask >> ((mybox * u) & 31)) & here);
            const int copies = __popc(__ballot_sync(0xFFFFFFFFu, mybox_seen));
            if (lane == 0) expect_bytes(bar, copies * u * kInner);
            __syncwarp();
            const int b = __shfl_sync(0xFFFFFFFFu, id, (from + mybox) & 31), p = __shfl_sync(0xFFFFFFFFu, place, (from + mybox) & 31);
            if (mybox_seen) {
                const uint32_t there = dst + h * (kTile * 128) + mybox * u * kInner;
                if (lane & 1) tma_load_4d(there + TT * Sh::kRowBytes, &a.v_map, h * 128, hk, p, b, bar);
                else tma_load_4d(there, &a.k_map, h * 128, hk, p, b, bar);
            }
        } else {
            const int64_t ko = at * a.cache.k_block + row * a.cache.k_token, vo = at * a.cache.v_block + row * a.cache.v_token;
            const char* kp = static_cast<const char*>(a.cache.k) + hk * a.cache.k_head;
            const char* vp = static_cast<const char*>(a.cache.v) + hk * a.cache.v_head;
            const int chunks = a.cache.dim / 16;
#pragma unroll 4
            for (int i = 0; i < TT * CH / 32; ++i) {
                const int r = (i * 32 + lane) / CH, ch = (i * 32 + lane) % CH;
                const int64_t kr = __shfl_sync(0xFFFFFFFFu, ko, r), vr = __shfl_sync(0xFFFFFFFFu, vo, r);
                const bool ok = ((mask >> r) & 1u) && ch < chunks;  // (past dim: zeros)
                const uint32_t there = dst + group_offset<CH>(r, ch);
                cp_async_16_zfill(there, ok ? kp + kr + ch * 16 : kp, ok);
                cp_async_16_zfill(there + TT * Sh::kRowBytes, ok ? vp + vr + ch * 16 : vp, ok);
            }
            if (lane == 0) expect_bytes(bar, 0);
        }
    }

    __device__ __forceinline__ bool arrived(int stage, uint32_t parity) const {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(bars + stage * 8), "r"(parity), "r"(100000u)
                     : "memory");
        return done != 0u;
    }
    // waits for a stage's tensor copies (cp.async: their groups), 0.8 s at most
    __device__ __forceinline__ void wait(int stage, uint32_t parity) {
        if (arrived(stage, parity)) return;
        for (int i = 0; !late && !arrived(stage, parity); ++i) late = i >= 8192;
    }
    // Whether a copy did not arrive.  Its row then starts no other, and what is on its way, from
    // stage `slot` on, is waited for here, 26 ms a stage at most: nothing of this warp is written
    // after it ends.  (Its results are worth nothing; all that follows stays in bounds.)
    __device__ __forceinline__ bool gave_up(int slot, uint32_t parity, int stages) {
        if (!__any_sync(0xFFFFFFFFu, late)) return false;
        if (!drained) {
            for (int i = 0; i < stages; ++i) {
                const int stage = slot + i < stages ? slot + i : slot + i - stages;
                for (int n = 0; n < 256 && !arrived(stage, stage >= slot ? parity : parity ^ 1u); ++n) {}
            }
            __syncwarp();
        }
        late = drained = true;
        return true;
    }
};

// Columns of a ring past dim are never copied: zeroed once.
__device__ __forceinline__ void clear_ring(uint8_t* smem, int bytes, int thread, int threads) {
    for (int i = thread; i < bytes / 16; i += threads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
}

template <int C>
__device__ __forceinline__ void store_lse(const Args<C>& a, int b, const Heads& hd, int h, float m, float l) {
    if (a.lse && h < hd.n) *lse_at<C>(a, b, hd, h) = lse_of<C>(m, l);
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
    template <int C>
    __device__ __forceinline__ void finish(const Args<C>& a, int b, const Heads& hd, int n, int k, int lane) const {
        const int r = lane >> 2, c = lane & 3;
        const float vs = C == kE4m3 ? a.cache.v_scale[hd.hk] : 1.f;
        const float f0 = l[0] != 0.f ? vs / l[0] : 0.f, f1 = l[1] != 0.f ? vs / l[1] : 0.f;
        const bool have = n * 8 + r < hd.n && k * 16 < a.cache.dim;
        store_dims<C>(o, f0, f1, have ? out_of<C>(a, b, hd, n * 8 + r) + k * 16 : nullptr, c);
        if (k == 0 && r == 0) {
            store_lse<C>(a, b, hd, n * 8 + 2 * c, m[0], l[0]);
            store_lse<C>(a, b, hd, n * 8 + 2 * c + 1, m[1], l[1]);
        }
    }
};

// The tiles [t0, t1) of one row, and where the row begins among all costs.
struct Segment {
    int at, b, row, t0, t1;
    Request q;
};

// Whether all of a CTA's W warps come after the one in which a row begins and before the one
// in which it ends.
template <int W>
__device__ __forceinline__ bool inside_of_row(int cta, int first, int last) {
    return first < cta * W && last >= (cta + 1) * W;
}

template <int C, int DP, int NT>
__global__ void __launch_bounds__((AttnShape<C, DP, NT>::kShareWarps * 32), 1)
    k_attention_shares(const __grid_constant__ Args<C> a, const JoinPlan jp) {
    using Sh = AttnShape<C, DP, NT>;
    constexpr int S = Sh::kStages, HEADS = Sh::kHeads, W = Sh::kShareWarps;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t tile_mask[W][S];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ring = smem_addr(smem) + warp * S * Sh::kStageBytes;
    const int rows = jp.rows;
    bool bad = false;

    GroupRing<C, DP, NT> groups;
    if constexpr (by_group(C)) {
        groups.open(a, smem_addr(smem), warp, W, S, lane);
        if (a.tensor_copies && threadIdx.x == 0) prefetch_tensor_map(&a.k_map), prefetch_tensor_map(&a.v_map);
    } else if (a.cache.dim != DP) {
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
    const bool may_team = by_group(C) && NT == 1 && jp.teams > 0;
    int count = may_team ? 1 : rows;  // rows that are counted of a request
    // the costs of requests base .. base + kScan - 1; returns those before this lane's, `sum`: all
    auto scan = [&](int base, int& sum) -> int {
        int own = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = base + lane * kPer + i;
            const int n = b < a.B ? request_of<C, Sh::kTokens>(a, b, bad).tiles : 0;
            cost[i] = n ? (n + kRowCost) * count : 0;
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
            const int n = request_of<C, Sh::kTokens>(a, b, bad).tiles;
            total += n ? (n + kRowCost) * count : 0;
        }
#pragma unroll
        for (int d = 16; d; d /= 2) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    }
    // teams: warps one after another have the same share of a request's rows, each of its own row,
    // so that `worker` counts along one row's warps, where that gives every warp kTeamTiles tiles
    // (16 requests of 0 to 4096 tokens, 3 tiles a warp: 24.5 us, without 23.0)
    const int place = blockIdx.x * W + warp;
    const bool teams = may_team && static_cast<int64_t>(total) * rows >= static_cast<int64_t>(kTeamTiles) * jp.warps;
    if (may_team && !teams) {
        count = rows;
        total *= rows, head_start *= rows;
#pragma unroll
        for (int i = 0; i < kPer; ++i) cost[i] *= rows;
    }
    const bool spare = teams && place >= jp.teams * rows;
    const int my_row = teams ? static_cast<unsigned>(place) % static_cast<unsigned>(rows) : 0;
    const int worker = teams && !spare ? my_row * jp.teams + place / rows : place;
    const int turn = teams ? (spare ? 0x7FFFFFFF : place / rows) : place;  // of the shares
    // requests without tokens
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (request_of<C, Sh::kTokens>(a, b, bad).tiles > 0) continue;
        if constexpr (by_group(C)) {
            const int per = a.cache.dim / 8;
            for (int i = threadIdx.x; i < a.tokens * a.q_heads * per; i += W * 32) {
                const int j = i / per, token = j / a.q_heads;
                *reinterpret_cast<uint4*>(a.out + b * a.out_request + token * a.out_token + (j - token * a.q_heads) * a.out_head + (i - j * per) * 8) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            if (a.lse)
                for (int j = threadIdx.x; j < a.tokens * a.q_heads; j += W * 32)
                    a.lse[static_cast<int64_t>(b) * a.tokens * a.q_heads + j] = -INFINITY;
        } else {
            store_empty<C>(a, b, Heads{0, 0, a.q_heads}, threadIdx.x, W * 32);
        }
        if (jp.by_row)
            for (int i = threadIdx.x; i < rows; i += W * 32) jp.joins[b * rows + i] = make_int4(-1, 0, 0, 0);
    }
    int workers = min((total + kMinCost - 1) / kMinCost, teams ? jp.teams : jp.warps);
    // one request: rows of one length, so a multiple of them splits none unevenly
    if (!teams && a.B == 1 && workers > rows) workers -= workers % rows;
    if (!jp.by_row && lane == 0) jp.joins[worker] = make_int4(-1, 0, 0, 0);
    if (turn >= workers) {
        if (bad) raise_device_error(a.err, W4A16_DEVERR_SLOT);
        return;
    }
    // costs before the i-th share: equal ones, the remainder to the first
    const unsigned share = static_cast<unsigned>(total) / static_cast<unsigned>(workers), extra = total - share * workers;
    const int u0 = turn * share + min(static_cast<unsigned>(turn), extra);
    const int u1 = u0 + share + (turn < static_cast<int>(extra) ? 1 : 0);
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
        if (teams || ++s.row == rows) {
            s.row = my_row;
            do {
                if (++s.b >= a.B) return false;
                s.q = request_of<C, Sh::kTokens>(a, s.b, bad);
            } while (s.q.tiles == 0);
        }
        open_segment(s);
        return true;
    };
    Segment seg{};
    bool live = u1 > u0 && locate(u0, seg.b, seg.at);
    if (live) {
        seg.q = request_of<C, Sh::kTokens>(a, seg.b, bad);
        if (teams) {
            seg.row = my_row;
        } else {
            seg.row = static_cast<unsigned>(u0 - seg.at) / static_cast<unsigned>(seg.q.tiles + kRowCost);
            seg.at += seg.row * (seg.q.tiles + kRowCost);
        }
        open_segment(seg);
        live = seg.t1 > seg.t0;
    }

    // Scales by group: a CTA all of whose warps lie inside of one row joins their parts itself, to
    // that of its first one, so that a long row leaves few to the join launch.
    __shared__ __align__(8) float near_ml[by_group(C) ? W : 1][2 * HEADS];
    bool inside = false;
    uint8_t* const rings = smem + (by_group(C) ? (0u - smem_addr(smem)) & 1023u : 0u);
    if constexpr (by_group(C))
        inside = live && !teams && inside_of_row<W>(blockIdx.x, worker_of(seg.at + kRowCost), worker_of(seg.at + kRowCost + seg.q.tiles - 1));

    // The copies run ahead of the products: `ahead` is the segment of the next
    // tile to copy, ahead_t the tile.
    RowMath<C, DP, NT> math;
    if (Sh::kQueries) math.queries = smem_addr(rings) + W * S * (Sh::kStageBytes + Sh::kBeside) + warp * Sh::kQueries;
    TileCopy<C, DP, NT> copy;
    Segment ahead = seg;
    int ahead_t = seg.t0, ahead_hk = heads_of<C, HEADS>(a, seg.row).hk;
    bool more = live;
    auto look_up = [&] {
        if constexpr (by_group(C)) groups.look_up(a, ahead.b, ahead_hk, ahead.q.tile0, ahead.q.start, ahead.q.len, ahead_t, ahead.t1, 1, lane);
        else copy.look_up(a, ahead.b, ahead.q, ahead_t, ahead.t1, 1, lane);
    };
    if (more) look_up();
    int t = seg.t0, put = 0, slot = 0, primed = 0;
    bool fresh = true;  // the next tile is the first of its row here
    Heads hd{};
    auto begin_row = [&] {
        // the queries are requested before the tiles, which they would queue behind
        fresh = false;
        hd = heads_of<C, HEADS>(a, seg.row);
        math.begin(a, seg.b, hd, lane);
        // and those of the row after this one brought to L2
        const bool same = !teams && seg.row + 1 < rows;
        const int after_b = same ? seg.b : seg.b + 1;
        if (after_b < a.B) {
            const Heads h = heads_of<C, HEADS>(a, same ? seg.row + 1 : my_row);
            constexpr int kLines = (DP + 63) / 64;
            for (int i = lane; i < h.n * kLines; i += 32)
                if ((i % kLines) * 64 < a.cache.dim) prefetch_l2(query_of<C>(a, after_b, h, i / kLines) + (i % kLines) * 64);
        }
    };
    // starts the copies of the next tile, if there is one
    auto copy_next = [&] {
        if (more) {
            if constexpr (by_group(C)) {
                if (a.scales != kTokenScales) groups.copy_boxes(a, ahead_hk, ahead.q, ahead_t, put, lane, bad);
                else groups.copy(a, ahead_hk, ahead.q, ahead_t, put, lane, bad);
            } else {
                const uint32_t mask = copy.copy(a, ahead_hk, ahead.q, ahead_t, 1, ring + put * Sh::kStageBytes, lane, bad);
                if (lane == 0) tile_mask[warp][put] = mask;
            }
            bool look = false;
            if (++ahead_t >= ahead.t1) {
                more = look = next_segment(ahead);
                ahead_t = ahead.t0;
                ahead_hk = heads_of<C, HEADS>(a, ahead.row).hk;
            }
            if constexpr (by_group(C)) look |= groups.known == 0;
            else look |= copy.wants(a, ahead_t, 1);
            if (more && look) look_up();
        }
        if (counts_groups<C>(a)) cp_async_commit();
        put = put + 1 == S ? 0 : put + 1;
    };
    // the row's tiles here are done: its result or its part
    auto end_row = [&] {
        math.reduce();
        const bool begins = seg.t0 == 0, ends = seg.t1 == seg.q.tiles;
        if (begins && ends) {
            math.finish(a, seg.b, hd, lane);
        } else {
            // (inside: into the ring, which is empty then)
            float* part = inside ? reinterpret_cast<float*>(rings + warp * S * Sh::kStageBytes)
                                 : jp.part + (static_cast<int64_t>(worker) * 2 + (begins ? 1 : 0)) * Sh::kPartFloats;
            float* const ml = inside ? near_ml[warp] : part + HEADS * DP;
            math.store_part(part, ml, ml + HEADS, lane);
        }
        // a row that begins here: what the join launch has to do for it
        if (begins && lane == 0 && (jp.by_row || !ends))
            jp.joins[jp.by_row ? seg.b * rows + seg.row : worker] =
                ends ? make_int4(-1, 0, 0, 0) : make_int4(seg.b, seg.row | (teams ? kTeamRow : 0), worker, worker - turn + worker_of(seg.at + kRowCost + seg.q.tiles - 1));
        live = next_segment(seg);
        t = seg.t0;
        fresh = true;
    };
    if constexpr (by_group(C)) {
        // A step works on the oldest tile and copies another into its place.  (S groups of
        // cp.async are on their way before it, empty ones among them.)
        uint32_t parity = 0u;
        while (live) {
            if (fresh) begin_row();
            for (; primed < S; ++primed) copy_next();
            if (counts_groups<C>(a)) cp_async_wait_group<S - 1>();
            groups.wait(slot, parity);
            if (groups.gave_up(slot, parity, S)) more = false;
            __syncwarp();  // (what the lanes themselves put into the stage)
            if (t == seg.t0) math.ready(a, seg.b, hd, seg.q.len, lane);
            math.tile(a, seg.q, groups.codes + slot * Sh::kStageBytes, groups.info + slot * Sh::kInfo, (seg.q.tile0 + t) * Sh::kTokens, lane);
            __syncwarp();
            copy_next();
            if (++slot == S) slot = 0, parity ^= 1u;
            if (++t >= seg.t1) end_row();
        }
        if (groups.late) raise_device_error(a.err, W4A16_DEVERR_TIMEOUT);
        if (inside) {
            __syncthreads();
            float* const out = jp.part + static_cast<int64_t>(blockIdx.x) * W * 2 * Sh::kPartFloats;
            for (int unit = threadIdx.x; unit < HEADS * DP / 4; unit += W * 32) {  // accumulator: (head block n, step k, lane)
                const int k = (unit >> 5) % Sh::kSteps, n = (unit >> 5) / Sh::kSteps, c = lane & 3;
                DimPart sum;
                sum.clear();
#pragma unroll 4
                for (int w = 0; w < W; ++w) {
                    const float* part = reinterpret_cast<const float*>(rings + w * S * Sh::kStageBytes);
                    const float2* ml = reinterpret_cast<const float2*>(near_ml[w]) + n * 4 + c;
                    sum.add(reinterpret_cast<const float4*>(part)[unit], ml[0], ml[HEADS / 2]);
                }
                reinterpret_cast<float4*>(out)[unit] = sum.o;
                if (k == 0 && lane < 4) {
                    float2* ml = reinterpret_cast<float2*>(out + HEADS * DP) + n * 4 + c;
                    ml[0] = make_float2(sum.m[0], sum.m[1]), ml[HEADS / 2] = make_float2(sum.l[0], sum.l[1]);
                }
            }
        }
    } else {
        // One step of the loop copies a tile and, once the ring is full, works on
        // the oldest one.
        while (live) {
            if (fresh) begin_row();
            const bool full = primed == S - 1;
            if (full) cp_async_wait_group<S - 2>();
            __syncwarp();
            copy_next();
            if (!full) {
                ++primed;
                continue;
            }
            if (t == seg.t0) math.ready(a, seg.b, hd, seg.q.len, lane);
            math.tile(ring + slot * Sh::kStageBytes, tile_mask[warp][slot], lane);
            slot = slot + 1 == S ? 0 : slot + 1;
            if (++t >= seg.t1) end_row();
        }
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

// Joins the parts of a row: grid (row, slice of its accumulators); threads
// (x: accumulators, y: group, of which each takes every n-th part, so that
// many parts are on their way at once).
constexpr int kJoinThreads = 512;  // at most
// parts a thread requests together (by group four: 24 requests, 20 heads of 64 dims 27.6 us with
// three or eight, 26.6)
constexpr int join_depth(int C, int NT) { return by_group(C) && NT == 1 ? 4 : 3; }

template <int C, int DP, int NT>
__global__ void __launch_bounds__(kJoinThreads) k_attention_join(const Args<C> a, const JoinPlan jp) {
    using Sh = AttnShape<C, DP, NT>;
    constexpr int HEADS = Sh::kHeads, KS = Sh::kSteps, kJoinDepth = join_depth(C, NT);
    __shared__ DimPart sums[kJoinThreads / 2];
    grid_dependents_launch();
    grid_dependency_wait();
    const int4 d = __ldcg(jp.joins + blockIdx.x);
    if (d.x < 0) return;
    const int unit = blockIdx.y * blockDim.x + threadIdx.x;  // accumulator: (head block n, step k, lane)
    const int lane = unit & 31, k = (unit >> 5) % KS, n = (unit >> 5) / KS, c = lane & 3;
    DimPart s;
    s.clear();
    // the i-th part: of warp first + i, where every CTA inside of the row has but one
    int parts = d.w - d.z + 1, lead = parts, inner = 0;  // warps before the CTAs inside; those CTAs
    if constexpr (by_group(C)) {
        constexpr int W = Sh::kShareWarps;
        const int from = d.z / W + 1;
        inner = d.y & kTeamRow ? 0 : max(d.w / W - from, 0);
        if (inner) {
            lead = from * W - d.z;
            parts -= inner * (W - 1);
        }
    }
    const auto warp_of = [&](int i) { return d.z + i + (i < lead ? 0 : min(i - lead, inner) * (Sh::kShareWarps - 1)); };
#pragma unroll 1
    for (int q = threadIdx.y; q < parts; q += blockDim.y * kJoinDepth) {
        float4 o[kJoinDepth];
        float2 m[kJoinDepth], l[kJoinDepth];
#pragma unroll
        for (int i = 0; i < kJoinDepth; ++i) {
            const int p = q + i * blockDim.y;
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            m[i] = l[i] = make_float2(0.f, 0.f);
            if (p < parts) {
                const float* part = jp.part + (static_cast<int64_t>(by_group(C) ? warp_of(p) : d.z + p) * 2 + (p == 0 ? 1 : 0)) * Sh::kPartFloats;
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
    s.finish<C>(a, d.x, heads_of<C, HEADS>(a, d.y & (kTeamRow - 1)), n, k, lane);
}

// kRowWarps / wpr rows per CTA, wpr warps for each; or (cluster > 1, wpr =
// kRowWarps) a row per cluster.  Tiles go round the CTAs of a row, then their
// warps.
template <int C, int DP, int NT>
__global__ void __launch_bounds__((AttnShape<C, DP, NT>::kRowWarps * 32), 1)
    k_attention_rows(const __grid_constant__ Args<C> a, const int rows, const int wpr, const int cluster) {
    using Sh = AttnShape<C, DP, NT>;
    constexpr int S = Sh::kRowStages, HEADS = Sh::kHeads, KS = Sh::kSteps, W = Sh::kRowWarps;
    extern __shared__ __align__(1024) uint8_t smem_all[];
    uint8_t* const smem = smem_all + (by_group(C) ? (0u - smem_addr(smem_all)) & 1023u : 0u);
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
    GroupRing<C, DP, NT> groups;
    if constexpr (by_group(C)) {
        groups.open(a, smem_addr(smem), warp, W, S, lane);
        if (a.tensor_copies && threadIdx.x == 0) prefetch_tensor_map(&a.k_map), prefetch_tensor_map(&a.v_map);
    } else if (a.cache.dim != DP) {
        clear_ring(smem, Sh::kRowSmem, threadIdx.x, W * 32);
        __syncthreads();
    }
    const Heads hd = b < a.B ? heads_of<C, HEADS>(a, row) : Heads{};
    grid_dependency_wait();
    grid_dependents_launch();
    // Queries, block ids (where they do not depend on the length) and length are
    // requested together.
    RowMath<C, DP, NT> math;
    if (Sh::kQueries) math.queries = smem_addr(smem) + W * S * (Sh::kStageBytes + Sh::kBeside) + warp * Sh::kQueries;
    TileCopy<C, DP, NT> copy;
    Request q{};
    if (b < a.B) {
        const bool early = a.window == 0 && (by_group(C) || TileCopy<C, DP, NT>::aligned(a));
        const int most_tiles = (a.most + Sh::kTokens - 1) / Sh::kTokens;
        if constexpr (by_group(C)) {
            if (early) groups.look_up(a, b, hd.hk, 0, 0, a.most, first_tile, most_tiles, step, lane);
        } else {
            if (early) copy.look_up(a, b, q, first_tile, most_tiles, step, lane);
        }
        math.begin(a, b, hd, lane);
        q = request_of<C, Sh::kTokens>(a, b, bad);
        if constexpr (by_group(C)) {
            if (!early) groups.look_up(a, b, hd.hk, q.tile0, q.start, q.len, first_tile, q.tiles, step, lane);
        } else {
            if (!early) copy.look_up(a, b, q, first_tile, q.tiles, step, lane);
        }
        if (q.tiles == 0 && rank == 0) store_empty<C>(a, b, hd, wir * 32 + lane, wpr * 32);
    }
    if (first_tile < q.tiles) {
        int ahead = first_tile, put = 0, slot = 0, primed = 0;
        auto copy_next = [&] {
            if (ahead < q.tiles) {
                if constexpr (by_group(C)) {
                    if (a.scales != kTokenScales) groups.copy_boxes(a, hd.hk, q, ahead, put, lane, bad);
                    else groups.copy(a, hd.hk, q, ahead, put, lane, bad);
                } else {
                    const uint32_t mask = copy.copy(a, hd.hk, q, ahead, step, ring + put * Sh::kStageBytes, lane, bad);
                    if (lane == 0) tile_mask[warp][put] = mask;
                }
                ahead += step;
                if constexpr (by_group(C)) {
                    if (ahead < q.tiles && groups.known == 0) groups.look_up(a, b, hd.hk, q.tile0, q.start, q.len, ahead, q.tiles, step, lane);
                } else {
                    if (ahead < q.tiles && copy.wants(a, ahead, step)) copy.look_up(a, b, q, ahead, q.tiles, step, lane);
                }
            }
            if (counts_groups<C>(a)) cp_async_commit();
            put = put + 1 == S ? 0 : put + 1;
        };
        if constexpr (by_group(C)) {
            uint32_t parity = 0u;
            for (; primed < S; ++primed) copy_next();
            for (int t = first_tile; t < q.tiles; t += step) {
                if (counts_groups<C>(a)) cp_async_wait_group<S - 1>();
                groups.wait(slot, parity);
                if (groups.gave_up(slot, parity, S)) ahead = q.tiles;
                __syncwarp();  // (what the lanes themselves put into the stage)
                if (t == first_tile) math.ready(a, b, hd, q.len, lane);
                math.tile(a, q, groups.codes + slot * Sh::kStageBytes, groups.info + slot * Sh::kInfo, (q.tile0 + t) * Sh::kTokens, lane);
                __syncwarp();
                copy_next();
                if (++slot == S) slot = 0, parity ^= 1u;
            }
            if (groups.late) raise_device_error(a.err, W4A16_DEVERR_TIMEOUT);
        } else {
            for (int t = first_tile; t < q.tiles;) {
                const bool full = primed == S - 1;
                if (full) cp_async_wait_group<S - 2>();
                __syncwarp();
                copy_next();
                if (!full) {
                    ++primed;
                    continue;
                }
                if (t == first_tile) math.ready(a, b, hd, q.len, lane);
                math.tile(ring + slot * Sh::kStageBytes, tile_mask[warp][slot], lane);
                slot = slot + 1 == S ? 0 : slot + 1;
                t += step;
            }
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
    const float vs = C == kE4m3 && joins ? a.cache.v_scale[hd.hk] : 1.f;
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
                    store_lse<C>(a, b, hd, h, m, l);
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
            store_dims<C>(o, f.x, f.y, n * 8 + r < hd.n && k * 16 < a.cache.dim ? out_of<C>(a, b, hd, n * 8 + r) + k * 16 : nullptr, c);
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
            if (rank == 0) store_lse<C>(a, b, hd, h, m, l);
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
        store_dims<C>(o, f.x, f.y, n * 8 + r < hd.n && k * 16 < a.cache.dim ? out_of<C>(a, b, hd, n * 8 + r) + k * 16 : nullptr, c);
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

template <int C, int DP, int NT>
cudaError_t launch_attention_shape(const Args<C>& all, const DeviceInfo& dev, JoinPlan jp, cudaStream_t s) {
    using Sh = AttnShape<C, DP, NT>;
    Args<C> a = all;
    int tokens = 1;
    if constexpr (by_group(C)) tokens = a.tokens;
    jp.rows = rows_of_request(a.q_heads * tokens, a.cache.heads, Sh::kHeads);
    int64_t all_rows = static_cast<int64_t>(a.B) * jp.rows;
    const int tiles = most_tiles(a.most, a.window > 0 ? a.window + tokens - 1 : 0, Sh::kTokens);  // of a row
    // short rows: as many warps for each as one wave of CTAs has, if that leaves
    // a warp few tiles
    {
        constexpr int W = Sh::kRowWarps;
        int wpr = W, cluster = 1;
        while (wpr > 1 && all_rows * wpr > static_cast<int64_t>(dev.sms) * W) wpr /= 2;
        // (19 tiles of 8 rows: 6.2 us with a CTA each, 6.9 with two, 5.9 with four)
        if (Sh::kClusters && wpr == W && tiles > kRowEnough * W)
            while (cluster < 8 && tiles > W * cluster && all_rows * cluster * 2 <= dev.sms) cluster *= 2;
        while (cluster > 1 && max_active_clusters(reinterpret_cast<const void*>(k_attention_rows<C, DP, NT>), W * 32,
                                                  Sh::kRowSmem, cluster) < all_rows)
            cluster /= 2;
        const int64_t grid = cluster > 1 ? all_rows * cluster : (all_rows * wpr + W - 1) / W;
        if (tiles <= kRowTiles * wpr * cluster)
            return launch_kernel(k_attention_rows<C, DP, NT>, true, cluster, dim3(static_cast<unsigned>(grid)), dim3(W * 32),
                                 Sh::kRowSmem, s, a, jp.rows, wpr, cluster);
    }
    const int ctas = std::min(dev.sms, most_workers(DP) / Sh::kShareWarps);
    jp.warps = ctas * Sh::kShareWarps;
    // Where a token's heads lie next to one another, the warps of an SM take the same tokens of all
    // of them at the same time.  One head after another would find the DRAM's pages closed again, at
    // a cost that differs between GPUs (64 requests of 8192 tokens of int8: 212 or 179 us, so 175 on
    // either; 24 of 12000 with 20 heads of 64 dims 215 or 190, so 155; where a block keeps each
    // head's tokens together 175 both ways).  Not where a row has so many warps that a CTA can join
    // theirs (one request of 131072 tokens: 60 or 54 us, so 58 or 57; of 32768 22, so 23), products
    // bound it (16 columns 72, 74), there is little for each warp, or many had nothing to do;
    // the kernel looks at what the lengths give.
    if constexpr (by_group(C) && NT == 1) {
        const int teams = jp.warps / jp.rows;
        const bool next_to = a.cache.k_head < a.cache.k_token && a.cache.v_head < a.cache.v_token;
        if (next_to && jp.rows > 1 && (jp.warps - teams * jp.rows) * 16 <= jp.warps && jp.warps < 128 * all_rows &&
            all_rows * (tiles + kRowCost) >= kTeamTiles * static_cast<int64_t>(jp.warps))
            jp.teams = teams;
    }
    // as many requests at a time as have costs of 32 bits (one has: attention_costs_fit)
    const int64_t fit = kMostCost / (static_cast<int64_t>(tiles + kRowCost) * jp.rows);
    for (int from = 0; from < all.B; from += a.B) {
        a.B = static_cast<int>(std::min<int64_t>(all.B - from, fit));
        a.q = all.q + from * a.q_request, a.out = all.out + from * a.out_request;
        a.block_table = all.block_table + from * a.table_stride, a.kv_len = all.kv_len + from;
        a.lse = all.lse ? all.lse + static_cast<int64_t>(from) * tokens * a.q_heads : nullptr;
        all_rows = static_cast<int64_t>(a.B) * jp.rows;
        jp.by_row = all_rows <= jp.warps;
        // (early, because a CTA has an SM for itself: several smaller ones that are placed
        // around others leave holes in the register file, and those that no longer fit then
        // run when the rest are done -- 20 key/value heads of 64 dims, 24 requests: 26 us)
        cudaError_t e = launch_kernel(k_attention_shares<C, DP, NT>, true, 1, dim3(ctas), dim3(Sh::kShareWarps * 32), Sh::kSmem,
                                      s, a, jp);
        if (e != cudaSuccess) return e;
        // few rows: their accumulators over several CTAs, down to a warp's; as many
        // groups as a row has parts for, if rows are alike
        const int places = jp.by_row ? static_cast<int>(all_rows) : jp.warps, units = Sh::kHeads * DP / 4;
        int width = 128;
        while (units % width || (width > 32 && places * (units / width) < dev.sms)) width /= 2;
        int parts = jp.warps / places + 2;
        if (by_group(C) && !jp.teams) parts = std::min(parts, 2 * Sh::kShareWarps + ctas / places);  // (a part a CTA inside of a row)
        int groups = 1;
        while (groups * width < kJoinThreads && groups * join_depth(C, NT) < parts) groups *= 2;
        e = launch_kernel(k_attention_join<C, DP, NT>, true, 1, dim3(places, units / width), dim3(width, groups), 0, s, a, jp);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Scales by group: more than 16 columns, which share what it takes to bring a tile and make
// it operands, as 24 or 32 together (16 requests of 16384 tokens at most, five new tokens of 4
// heads: as 16 and 4 96 us, as 24 77).
template <int C>
cudaError_t launch_attention_wide(const Args<C>& a, const DeviceInfo& dev, const JoinPlan& jp, cudaStream_t s) {
    const bool three = columns_together(a.q_heads / a.cache.heads * a.tokens, a.cache.dim) == 24;
    switch (padded_dim(a.cache.dim)) {
        case 64: return three ? launch_attention_shape<C, 64, 3>(a, dev, jp, s) : launch_attention_shape<C, 64, 4>(a, dev, jp, s);
        case 96: return three ? launch_attention_shape<C, 96, 3>(a, dev, jp, s) : launch_attention_shape<C, 96, 4>(a, dev, jp, s);
        default: return three ? launch_attention_shape<C, 128, 3>(a, dev, jp, s) : launch_attention_shape<C, 128, 4>(a, dev, jp, s);
    }
}

template <int C>
cudaError_t launch_attention_type(const Args<C>& a, const DeviceInfo& dev, const JoinPlan& jp, cudaStream_t s) {
    int tokens = 1;
    if constexpr (by_group(C)) tokens = a.tokens;
    const bool wide = a.q_heads / a.cache.heads * tokens > 8;
    // 16 heads of 256 dims fill a warp's registers: two rows of 8 are faster while the second
    // finds the cache in L2 (8 requests, windows of 4096: 15.4 us against 18.0; 134 MB over
    // e4m3 50 against 58; but 1.07 GB of bf16 328 against 216)
    const int64_t visible = a.window > 0 && a.window < a.most ? a.window : a.most;
    const bool in_l2 = static_cast<double>(a.B) * visible * a.cache.heads * a.cache.dim * (in_8_bits(C) ? 2 : 4) <= (1 << 27);
    switch (padded_dim(a.cache.dim)) {
        case 64: return wide ? launch_attention_shape<C, 64, 2>(a, dev, jp, s) : launch_attention_shape<C, 64, 1>(a, dev, jp, s);
        case 96: return wide ? launch_attention_shape<C, 96, 2>(a, dev, jp, s) : launch_attention_shape<C, 96, 1>(a, dev, jp, s);
        case 128: return wide ? launch_attention_shape<C, 128, 2>(a, dev, jp, s) : launch_attention_shape<C, 128, 1>(a, dev, jp, s);
        case 192: return wide ? launch_attention_shape<C, 192, 2>(a, dev, jp, s) : launch_attention_shape<C, 192, 1>(a, dev, jp, s);
        default: return wide && !in_l2 ? launch_attention_shape<C, 256, 2>(a, dev, jp, s) : launch_attention_shape<C, 256, 1>(a, dev, jp, s);
    }
}

}  // namespace
}  // namespace w4a16
