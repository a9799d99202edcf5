// What the two launches of w4a16_paged_attention share.  Internal to the library.
#pragma once

#include "paged.h"

namespace w4a16 {

constexpr int kMostAttnCtas = 320;  // of the first launch: two on each of 152 SMs, rounded up

// Over an e4m3 cache the probabilities go into fp16 products as 2^15 p: fp16
// then holds them down to 2^-39 of the largest.  The factor leaves again with
// the division by their sum.
constexpr float kE4m3Bias = 15.f;

// Rows that several CTAs of the first launch share, for the second to join.
struct JoinPlan {
    // {request or -1: nothing to join, row of the request, first CTA, last CTA}: one per
    // row (by_row: no more rows than CTAs), else one per CTA, for the row that begins in
    // it and goes on in the next
    int4* joins;
    // [cta][2][heads * (padded + 2)]: o [heads][padded], m [heads] (log2 units), l [heads];
    // place 0: the row that the CTA's share begins inside of, 1: the row it ends inside of
    float* part;
    int by_row;
    int split;   // rows may span CTAs: the second launch is needed
    int rows;    // of a request: key/value heads times chunks of the query heads sharing one
    int heads;   // query heads of a chunk: 8 or 16
    int padded;  // dim rounded up to 64
    int ctas;    // of the first launch
};

// paged_attention_bf16.cu, paged_attention_e4m3.cu: the first launch; fills in the plan
cudaError_t launch_attention_bf16(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan& join, cudaStream_t s);
cudaError_t launch_attention_e4m3(const AttentionArgs& a, const DeviceInfo& dev, JoinPlan& join, cudaStream_t s);

}  // namespace w4a16
