// What the launches of w4a16_paged_attention share.  Internal to the library.
#pragma once

#include "paged.h"

namespace w4a16 {

// Over an e4m3 cache the probabilities go into fp16 products as 2^15 p: fp16
// then holds them down to 2^-39 of the largest.  The factor leaves again with
// the division by their sum.
constexpr float kE4m3Bias = 15.f;

// The dims a kernel is built for: dim rounded up to one of them.
constexpr int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }

// Most warps of the first launch, by the padded dim: 16, 12 or 8 on each of up
// to 160 SMs.
constexpr int most_workers(int padded) { return padded == 64 ? 2560 : padded <= 128 ? 1920 : 1280; }

constexpr int kTile = 16;    // tokens of a tile: the MMA's rows
constexpr int kRowCost = 2;  // a row's queries and result, in tiles (1: 128 requests over e4m3 132 us, 2: 125)
constexpr int kMostCost = 0x7FFFFF00;  // of all rows of a launch: sums a little above it still fit 32 bits

// Tiles of a row at most (a window may begin inside one).
constexpr int most_tiles(int most, int window, int tokens = kTile) {
    const int visible = window > 0 && window < most ? window : most;
    return (visible + tokens - 1) / tokens + (visible < most);
}
// Rows of a request: `heads` query heads of a key/value head, or fewer, each.
constexpr int rows_of_request(int q_heads, int kv_heads, int heads) {
    return kv_heads * ((q_heads / kv_heads + heads - 1) / heads);
}

// Rows that several warps of the first launch share, for the second to join.
// A part is what a warp has of a row: o as the products' accumulators hold it
// (float4 per lane and 16 dims), then m (log2 units) and l of each head.
struct JoinPlan {
    // {request or -1: nothing to join, row of the request (marked by kTeamRow where every warp
    // left a part), first warp, last warp}: one per row (by_row: no more rows than warps), else
    // one per warp, for the row that begins in it and goes on in the next
    int4* joins;
    // [warp][2][heads * (padded + 2)]; place 0: the row that the warp's share begins inside
    // of, 1: the row it ends inside of
    float* part;
    int by_row;
    int rows;   // of a request: key/value heads times chunks of the query heads sharing one
    int warps;  // of the first launch
    int teams;  // by group: 0, or how many warps share each row of a request, the same shares for all of its rows
};

// paged_attention_bf16.cu, paged_attention_e4m3.cu: all launches of a call; `join` has joins and part
cudaError_t launch_attention_bf16(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);
cudaError_t launch_attention_e4m3(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan join, cudaStream_t s);

}  // namespace w4a16
