// Host-side launcher interface of the operators over a w4a16_scaled_cache
// (append that finds the scales, read, attention).  Internal to the library.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "paged.h"

namespace w4a16 {

constexpr int kMostGroup = 128;  // tokens of a scale
constexpr int kMostNew = 16;     // new tokens of a request

// place / group for places of a page (below 2^16) by one multiplication: the high
// half of place * ceil(2^32 / group).  (0 stands for a group of one.)
inline uint32_t group_magic(int group) {
    return group == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + group - 1) / group);
}

struct ScaledAppendArgs {
    const uint16_t* q;
    uint16_t* q_out;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_token, q_head, qo_token, qo_head, k_token, k_head, v_token, v_head;
    const int32_t* positions;
    int64_t axis_stride;
    const float* inv_freq;
    int axis_end[4];  // pairs below axis_end[a] (and not below axis_end[a - 1]) go by axis a
    const int32_t* slots;
    w4a16_scaled_cache cache;
    int q_heads;  // 0 where there are no queries
    int rotary;
    int dim;
    int interleaved;
    int64_t T;
    uint32_t* err;
};

cudaError_t launch_scaled_append(const ScaledAppendArgs& a, const DeviceInfo& dev, cudaStream_t s);

struct ScaledReadArgs {
    w4a16_scaled_cache cache;
    const int32_t* block_table;
    int64_t table_stride;
    const int32_t* row_start;
    const int32_t* first;  // NULL: 0
    void* k_out;
    void* v_out;
    int64_t k_row, k_out_head, v_row, v_out_head;
    int64_t rows;
    int columns;
    int B;
    int out_f32;
    uint32_t* err;
};

cudaError_t launch_scaled_read(const ScaledReadArgs& a, const DeviceInfo& dev, cudaStream_t s);

constexpr int kBoxScales = 0;    // a box lies in one group, whose scales come with its block id
constexpr int kRowScales = 1;    // groups of 1, 2 or 4 tokens, four or more in a box, their scales one after another in memory
constexpr int kTokenScales = 2;  // one by one

// The one-token launch's arguments (its cache without scales; q_heads: those of a
// token), and what several tokens and scales by group need.
struct ScaledAttentionArgs : AttentionArgs {
    int tokens;  // new ones of a request
    int64_t q_token, out_token;
    const float* k_scale;
    const float* v_scale;
    int64_t ks_block, ks_group, ks_head, vs_block, vs_group, vs_head;
    int group;
    uint32_t magic;  // of group
    // A tile's tokens are boxes of 2^box_log2, each in one block; tensor_copies: their codes come by
    // tensor copies (boxes of 8, 16 or 32 tokens).
    int box_log2, tensor_copies;
    int scales;      // where those of a tile come from:
    int group_log2;  //   kRowScales: of group; else 0
    CUtensorMap k_map;  // boxes of one head's values by `box` tokens of a block
    CUtensorMap v_map;
};

// The tensor map of keys or values: boxes of `inner` codes (64 or 128, their swizzle) of a
// head by `box` tokens of a block; codes past dim read as zeros.  False where there is none
// for these strides.
bool encode_cache_map(CUtensorMap* map, const void* codes, const w4a16_scaled_cache& c, int64_t block, int64_t token, int64_t head, int inner,
                      int box);

// Columns (new tokens times the query heads of a key/value head) that are worked on together:
// 8, 16, and up to 128 dims 24 or 32, of as equal rows as there are.
constexpr int most_together(int dim) { return dim <= 128 ? 32 : 16; }
constexpr int columns_together(int columns, int dim) {
    const int most = most_together(dim), rows = (columns + most - 1) / most;
    return (columns + 8 * rows - 1) / (8 * rows) * 8;
}
size_t scaled_attention_workspace(int q_heads, int kv_heads, int dim, int new_tokens);
cudaError_t launch_scaled_attention(const ScaledAttentionArgs& a, int int8, const DeviceInfo& dev, cudaStream_t s);

}  // namespace w4a16
