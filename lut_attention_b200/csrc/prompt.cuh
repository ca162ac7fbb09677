// Packed prompts: where each sequence's queries and keys lie, and which tile of
// queries a CTA takes.  The starts are device memory; every value is clamped to
// the packed extents, so that wrong starts give wrong rows but no access outside
// the tensors.
#pragma once

#include <cstdint>

#include "bounds.cuh"

namespace axr {

struct PromptShape {
    const int32_t *cu_q, *cu_k;        // batch + 1 starts
    int batch;
    int heads, group;
    int total_q, total_k;
    int64_t q_head, q_row, k_head, k_row, v_head, v_row, o_head, o_row;   // strides in elements
};

struct PromptArgs {
    const void *q, *K, *V;
    int dtype;
    int d;
    PromptShape s;
    void *out;
    float *lse;                        // (heads*group, total_q), or null
};

struct PromptTile {
    int first_q, len_q;                // the sequence's queries
    int first_k, len_k;                // and keys
    int row;                           // first query of the tile in the sequence
};

// tiles of `bm` queries that `batch` sequences of `total_q` queries can have at most
inline int prompt_tiles(const PromptShape &s, int bm)
{
    const int64_t full = s.total_q / bm, ragged = s.batch < s.total_q ? s.batch : s.total_q;
    return static_cast<int>(full + ragged);
}

// The tile of BM queries that comes `index`-th over all sequences, the last
// tiles of a sequence first (they see the most keys, so the grid's tail is its
// short ones); false past the last.  Called by whole warps with the same index.
template <int BM>
__device__ __forceinline__ bool find_tile(const PromptShape &s, int index,
                                          PromptTile &t AXR_DEBUG_ONLY(, const dbg::Span &sp_q, const dbg::Span &sp_k))
{
    const int lane = threadIdx.x & 31;
    auto start = [&](const int32_t *cu, int i, int total AXR_DEBUG_ONLY(, const dbg::Span &sp)) {
        const int v = AXR_IN(sp, cu + i, 4) ? cu[i] : 0;
        return min(max(v, 0), total);
    };
    for (int b0 = 0; b0 < s.batch; b0 += 32) {
        const int b = b0 + lane;
        int first = 0, len = 0;
        if (b < s.batch) {
            first = start(s.cu_q, b, s.total_q AXR_DEBUG_ONLY(, sp_q));
            len = max(0, start(s.cu_q, b + 1, s.total_q AXR_DEBUG_ONLY(, sp_q)) - first);
        }
        const int tiles = (len + BM - 1) / BM;
        int upto = tiles;                                     // inclusive scan over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, index < upto);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int before = __shfl_sync(0xffffffffu, upto - tiles, src);
            const int n = __shfl_sync(0xffffffffu, tiles, src);
            t.first_q = __shfl_sync(0xffffffffu, first, src);
            t.len_q = __shfl_sync(0xffffffffu, len, src);
            t.row = (n - 1 - (index - before)) * BM;
            t.first_k = start(s.cu_k, b0 + src, s.total_k AXR_DEBUG_ONLY(, sp_k));
            t.len_k = max(0, start(s.cu_k, b0 + src + 1, s.total_k AXR_DEBUG_ONLY(, sp_k)) - t.first_k);
            return true;
        }
        index -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

}  // namespace axr
