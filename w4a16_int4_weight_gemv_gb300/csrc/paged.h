// Host-side launcher interface of the paged-cache operators (block map,
// rotary + cache append, one-token attention).  Internal to the library.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "launch.h"
#include "w4a16.h"

namespace w4a16 {

struct PagedMapArgs {
    const int32_t* ctx_len;
    const int32_t* new_len;
    int32_t* block_table;
    int64_t table_stride;
    const int32_t* free_blocks;
    const int32_t* free_head;
    int32_t* slots;
    int32_t* positions;
    int32_t* row_start;
    int32_t* kv_len;
    int32_t* free_head_out;
    int64_t n_free;
    int64_t num_blocks;
    int64_t tokens;
    int B;
    int columns;
    int page;
    uint32_t* err;
};

constexpr int kMaxMapRequests = 16384;  // three prefix arrays of this length fit shared memory

cudaError_t launch_paged_map(const PagedMapArgs& a, const DeviceInfo& dev, cudaStream_t s);

struct RopeArgs {
    const uint16_t* q;
    uint16_t* q_out;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_token, q_head, qo_token, qo_head, k_token, k_head, v_token, v_head;
    const int32_t* positions;
    int64_t axis_stride;
    const float* inv_freq;
    int axes;
    int axis_end[4];  // pairs below axis_end[a] (and not below axis_end[a - 1]) go by axis a
    const int32_t* slots;
    w4a16_kv_cache cache;  // heads 0 where there is none
    int q_heads;
    int rotary;
    int dim;
    int interleaved;
    int inverse;
    int64_t T;
    uint32_t* err;
};

cudaError_t launch_rope_append(const RopeArgs& a, const DeviceInfo& dev, cudaStream_t s);

struct AttentionArgs {
    const uint16_t* q;
    int64_t q_request, q_head;
    w4a16_kv_cache cache;
    const int32_t* block_table;
    int64_t table_stride;
    const int32_t* kv_len;
    int most;  // tokens a row of the table holds
    int B;
    int q_heads;
    int window;
    float scale;
    uint16_t* out;
    int64_t out_request, out_head;
    float* lse;
    void* workspace;
    uint32_t* err;
};

// Whether the tiles that one request can have fit the 32 bits in which the launch
// counts them.
bool attention_costs_fit(int most, int window, int q_heads, int kv_heads);

size_t paged_attention_workspace(int q_heads, int kv_heads, int dim);
cudaError_t launch_paged_attention(const AttentionArgs& a, const DeviceInfo& dev, cudaStream_t s);

}  // namespace w4a16
