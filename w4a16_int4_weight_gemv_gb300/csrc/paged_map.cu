// Block tables and slot maps from request lengths (w4a16_paged_map).
//
// Both outputs follow from two exclusive prefix sums over the requests: of
// the new tokens (where a request's slots begin) and of the new blocks (where
// its share of the free list begins).  Every CTA forms both sums itself --
// 8 bytes a request, from L2 -- and then takes its share of the tokens and
// of the table entries, finding a token's request by bisection in shared
// memory.  So one launch does it all, no CTA waits for another, and an entry
// of the table that this call writes is never one that it reads: tokens in a
// request's half-filled last block read an old entry, tokens in new blocks
// take the id from the free list as the entry's writer does.
//
// Bound by latency (length, sums, table entry, store): on one GB300, in a CUDA
// graph, 2.9 us for 16 requests of one new token, 4.9 us for 262144 tokens of 96
// requests, whose 2.3 MB would take 0.34 us (3.2 and 5.2 us a call).  (A launch
// for the sums and one for the rest would cost a launch more; 512 threads a CTA,
// 7.7 us for the latter case.)
#include "common.cuh"
#include "paged.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;

struct Pair {
    int64_t tokens, blocks;
};

__device__ __forceinline__ Pair warp_inclusive(Pair v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v.tokens, d);
        const int64_t b = __shfl_up_sync(0xFFFFFFFFu, v.blocks, d);
        if (lane >= d) {
            v.tokens += t;
            v.blocks += b;
        }
    }
    return v;
}

__device__ __forceinline__ int clamp_i32(int64_t v) {
    return v > 0x7FFFFFFF ? 0x7FFFFFFF : static_cast<int>(v);
}

// the last request whose first item is at or before i (start[] ascending, start[0] = 0)
__device__ __forceinline__ int owner_of(const int* start, int n, int i) {
    int lo = 0, hi = n;  // start[lo] <= i < start[hi] (past the end: none)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// PER: consecutive tokens of a thread, which mostly lie in one block.
template <int PER>
__global__ void __launch_bounds__(kThreads) k_paged_map(const PagedMapArgs a) {
    extern __shared__ int sm[];
    int* tok = sm;                // [B + 1] new tokens before request b
    int* blk = sm + a.B + 1;      // [B + 1] new blocks before request b
    int* ctx = sm + 2 * a.B + 2;  // [B] cached tokens
    __shared__ Pair warp_sum[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool first_cta = blockIdx.x == 0;
    uint32_t bad = 0u;

    grid_dependency_wait();
    grid_dependents_launch();
    Pair carry{0, 0};
    for (int base = 0; base < a.B; base += kThreads) {
        const int b = base + static_cast<int>(threadIdx.x);
        Pair mine{0, 0};
        int c = 0;
        if (b < a.B) {
            int n = a.new_len[b];
            c = a.ctx_len[b];
            if (c < 0 || n < 0) bad |= W4A16_DEVERR_BLOCKS;
            c = max(c, 0);
            n = max(n, 0);
            const int64_t end = static_cast<int64_t>(c) + n;
            const int64_t before = min((static_cast<int64_t>(c) + a.page - 1) / a.page,
                                       static_cast<int64_t>(a.columns));
            int64_t after = (end + a.page - 1) / a.page;
            if (after > a.columns) {
                bad |= W4A16_DEVERR_BLOCKS;
                after = a.columns;
            }
            mine = Pair{n, after - before};
            if (first_cta) a.kv_len[b] = clamp_i32(end);
        }
        const Pair inc = warp_inclusive(mine, lane);
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        Pair before_warp = carry, total = carry;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) {
                before_warp.tokens += warp_sum[w].tokens;
                before_warp.blocks += warp_sum[w].blocks;
            }
            total.tokens += warp_sum[w].tokens;
            total.blocks += warp_sum[w].blocks;
        }
        if (b < a.B) {
            const int t0 = clamp_i32(before_warp.tokens + inc.tokens - mine.tokens);
            tok[b] = t0;
            blk[b] = clamp_i32(before_warp.blocks + inc.blocks - mine.blocks);
            ctx[b] = c;
            if (first_cta) a.row_start[b] = t0;
        }
        carry = total;
        __syncthreads();
    }
    const int64_t head = *a.free_head;
    if (threadIdx.x == 0) {
        tok[a.B] = clamp_i32(carry.tokens);
        blk[a.B] = clamp_i32(carry.blocks);
        if (first_cta) {
            a.row_start[a.B] = clamp_i32(carry.tokens);
            *a.free_head_out = clamp_i32(min(head + carry.blocks, max(a.n_free, head)));
            if (carry.tokens > a.tokens || head < 0 || head + carry.blocks > a.n_free)
                bad |= W4A16_DEVERR_BLOCKS;
        }
    }
    __syncthreads();

    // new block i of all: the free list's entry head + i, or -1
    auto fresh_block = [&](int i) -> int {
        const int64_t at = head + i;
        if (head < 0 || at >= a.n_free) return -1;
        const int id = a.free_blocks[at];
        if (id >= 0 && id < a.num_blocks) return id;
        bad |= W4A16_DEVERR_SLOT;
        return -1;
    };
    const int step = static_cast<int>(gridDim.x) * kThreads;
    const int me = static_cast<int>(blockIdx.x) * kThreads + static_cast<int>(threadIdx.x);

    const int nblk = blk[a.B];
    for (int64_t i = me; i < nblk; i += step) {
        const int b = owner_of(blk, a.B, static_cast<int>(i));
        const int64_t before = (static_cast<int64_t>(ctx[b]) + a.page - 1) / a.page;
        a.block_table[b * a.table_stride + before + (i - blk[b])] = fresh_block(static_cast<int>(i));
    }

    const int ntok = tok[a.B];
    const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
    for (int64_t t0 = static_cast<int64_t>(me) * PER; t0 < a.tokens; t0 += static_cast<int64_t>(step) * PER) {
        int pos[PER], slot[PER];
        int b = t0 < ntok ? owner_of(tok, a.B, static_cast<int>(t0)) : 0, of_b = -1, of_col = -1, id = -1;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int64_t t = t0 + j;
            pos[j] = slot[j] = -1;
            if (t >= ntok) continue;
            while (t >= tok[b + 1]) ++b;
            pos[j] = clamp_i32(static_cast<int64_t>(ctx[b]) + (t - tok[b]));
            const int col = static_cast<int>(static_cast<unsigned>(pos[j]) / static_cast<unsigned>(a.page));
            if (b != of_b || col != of_col) {
                of_b = b, of_col = col, id = -1;
                const int before = static_cast<int>((static_cast<int64_t>(ctx[b]) + a.page - 1) / a.page);
                if (col < a.columns) {
                    if (col < before) {
                        id = a.block_table[b * a.table_stride + col];
                        if (id < 0 || id >= a.num_blocks) {
                            id = -1;
                            bad |= W4A16_DEVERR_SLOT;
                        }
                    } else {
                        id = fresh_block(blk[b] + (col - before));
                    }
                }
            }
            if (id >= 0) slot[j] = static_cast<int>(static_cast<int64_t>(id) * a.page + (pos[j] - col * a.page));
        }
        if (PER == 4 && wide && t0 + PER <= a.tokens) {
            *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[PER > 1], pos[PER > 2 ? 2 : 0], pos[PER > 3 ? 3 : 0]);
            *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[PER > 1], slot[PER > 2 ? 2 : 0], slot[PER > 3 ? 3 : 0]);
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (t0 + j < a.tokens) {
                    a.positions[t0 + j] = pos[j];
                    a.slots[t0 + j] = slot[j];
                }
        }
    }
    if (bad) raise_device_error(a.err, bad);
}

}  // namespace

cudaError_t launch_paged_map(const PagedMapArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    // a token a thread while two CTAs an SM hold them, else four (262144 tokens of 96
    // requests: 6.1 us with one, 5.0 with four)
    const int64_t most = 2LL * dev.sms * kThreads;
    const bool many = a.tokens > most;
    auto* kernel = many ? k_paged_map<4> : k_paged_map<1>;
    const int smem = (3 * a.B + 2) * static_cast<int>(sizeof(int));
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    const int64_t per_cta = kThreads * (many ? 4 : 1);
    int64_t ctas = (a.tokens + per_cta - 1) / per_cta;
    if (ctas > 2 * dev.sms) ctas = 2 * dev.sms;
    if (ctas < 1) ctas = 1;
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
    const cudaError_t rc = cudaLaunchKernelEx(&cfg, kernel, a);
    return rc != cudaSuccess ? rc : cudaGetLastError();
}

}  // namespace w4a16
