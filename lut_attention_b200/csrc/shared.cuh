// Decode attention over a shared quantized prefix and each sequence's own
// quantized keys: the split of the work that the kernels share.
//
// The work is a list of segments, each a block of queries against one run of
// keys: per KV head (and block of BM of its batch * group queries) the prefix,
// then per sequence and KV head its own keys against its `group` queries.  A
// segment is cut into tiles of 128 keys; all segments form one line, in which
// each stands for run_cost places (what taking up its queries and writing its sums
// costs, in tiles) and then one place a tile.  CTA c of C takes an equal stretch of
// the line.  Where it leaves a segment (or its stretch ends) it writes the queries'
// running (o, m, l) to a slot of the workspace.  Along the line every step to
// another slot raises the segment or the CTA, so segment + CTA numbers the slots
// without a table.  The last kernel merges the slots of each query.  The split
// depends on the lengths alone, so results repeat bit for bit.
#pragma once

#include <cstdint>

#include "axr_internal.cuh"

namespace axr {
namespace shared {

constexpr int kTileKeys = 128;

// What every kernel of a call gets.
struct Work {
    const int32_t *lengths;            // (batch): own keys of each sequence, clamped to [0, capacity]
    int n;                             // prefix keys
    int capacity;
    int batch, heads, group;
    int d;
    int bm;                            // queries of a prefix segment
    int row_tiles;                     // ceil(batch * group / bm)
    int slot_rows;                     // rows of a prefix slot: min(bm, batch * group)
    int ctas;                          // CTAs of the main kernel (at most)
    int run_cost;                      // places of a segment before its tiles
    // workspace
    void *rot;                         // rotated queries: batch * heads * group rows of d 32-bit words
    float *rot_scale;                  // one factor per query (tensor-core kernel)
    int32_t *own_start;                // (batch + 1): places of the own keys of sequences before b, per KV head
    float *prefix_part;                // (heads * row_tiles + ctas) slots of slot_rows x (d + 2): o, m, l
    float *own_part;                   // (batch * heads + ctas) slots of group x (d + 2)
    AXR_DEBUG_ONLY(dbg::Span sp_lengths, sp_rot, sp_rot_scale, sp_own_start, sp_prefix_part, sp_own_part;)
};

struct Line {
    int prefix_places;                 // per prefix segment, 0 without a prefix
    int own_first;                     // first place of the own segments
    int total;                         // below 2^31 (checked on the host)
    int ctas;                          // that take part
    __device__ int begin(int c) const { return share(total, c, 0, ctas); }
    // the CTA that holds place t
    __device__ int owner(int t) const { return share(t + 1, ctas, 1, total); }
    // (a * b - less) / c; in 32 bits, several times as fast, where all such products fit
    __device__ int share(int a, int b, int less, int c) const
    {
        if (total <= INT32_MAX / ctas) return (a * b - less) / c;
        return static_cast<int>((static_cast<int64_t>(a) * b - less) / c);
    }
};

// places of a segment of `keys` keys
__device__ __forceinline__ int places(const Work &w, int keys)
{
    return keys > 0 ? w.run_cost + (keys + kTileKeys - 1) / kTileKeys : 0;
}

__device__ __forceinline__ int own_start(const Work &w, int b)
{
    return AXR_IN(w.sp_own_start, w.own_start + b, 4) ? w.own_start[b] : 0;
}

// own: places of all sequences' own keys, per KV head
__device__ __forceinline__ Line line_of(const Work &w, int own)
{
    Line x;
    x.prefix_places = places(w, w.n);
    x.own_first = w.heads * w.row_tiles * x.prefix_places;
    x.total = x.own_first + w.heads * own;
    // small calls take as many CTAs as stretches of two places give
    x.ctas = min(max(x.total / 2, 1), w.ctas);
    return x;
}

// A run of tiles of one segment.
struct Run {
    int head, seq;                     // KV head; sequence, or -1 for the prefix
    int row0, rows;                    // prefix: queries row0 .. of the head's batch * group; own: 0, group
    int tile, tiles;                   // tiles [tile, tile + tiles) of the segment; none if only its other places are met
    int keys;                          // keys of the segment
    int seg;                           // segment number among the prefix or own segments
    int next;                          // the place after it: the segment's end or the stretch's
    // its first key row
    __device__ int64_t base(const Work &w) const
    {
        return seq >= 0 ? static_cast<int64_t>(seg) * w.capacity : static_cast<int64_t>(head) * w.n;
    }
};

// own keys of sequence b
__device__ __forceinline__ int length(const Work &w, int b)
{
    const int len = AXR_IN(w.sp_lengths, w.lengths + b, 4) ? w.lengths[b] : 0;
    return min(max(len, 0), w.capacity);
}

// The run at place t of a stretch that ends at `end`; start(b) is own_start of
// sequence b, keys(b) its length.
template <typename Start, typename Keys>
__device__ __forceinline__ Run run_at(const Work &w, const Line &x, int t, int end, Start start, Keys keys)
{
    Run r;
    int first, per;                                           // the segment's first place, and its places
    if (t < x.own_first) {
        r.seg = t / x.prefix_places;
        per = x.prefix_places;
        first = r.seg * per;
        r.head = r.seg / w.row_tiles;
        r.seq = -1;
        r.row0 = r.seg % w.row_tiles * w.bm;
        r.rows = min(w.bm, w.batch * w.group - r.row0);
        r.keys = w.n;
    } else {
        const int u = t - x.own_first;
        int lo = 0, hi = w.batch;                             // the last b with heads * own_start[b] <= u
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (w.heads * start(mid) <= u) lo = mid;
            else hi = mid;
        }
        const int s0 = start(lo);
        per = start(lo + 1) - s0;
        r.head = (u - w.heads * s0) / per;
        first = x.own_first + w.heads * s0 + r.head * per;
        r.seq = lo;
        r.row0 = 0;
        r.rows = w.group;
        r.keys = keys(lo);
        r.seg = lo * w.heads + r.head;
    }
    r.next = min(first + per, end);
    const int from = max(t, first + w.run_cost);              // the first tile's place
    r.tile = from - first - w.run_cost;
    r.tiles = max(r.next - from, 0);
    return r;
}

// the query row (of batch * heads * group) of row i of a run
__device__ __forceinline__ int64_t query_row(const Work &w, const Run &r, int i)
{
    if (r.seq >= 0) return static_cast<int64_t>(r.seg) * w.group + i;
    const int at = r.row0 + i;
    return (static_cast<int64_t>(at / w.group) * w.heads + r.head) * w.group + at % w.group;
}

// where row i of a run writes its (o[d], m, l)
__device__ __forceinline__ float *slot(const Work &w, const Run &r, int cta, int i)
{
    if (r.seq >= 0) return w.own_part + (static_cast<int64_t>(r.seg + cta) * w.group + i) * (w.d + 2);
    return w.prefix_part + (static_cast<int64_t>(r.seg + cta) * w.slot_rows + i) * (w.d + 2);
}

__device__ __forceinline__ Run run_at(const Work &w, const Line &x, int t, int end)
{
    return run_at(w, x, t, end, [&](int b) { return own_start(w, b); }, [&](int b) { return length(w, b); });
}

// places of a call at most (own keys: all of capacity), or more than 2^31 - 1
inline int64_t most_places(const Work &w)
{
    const auto of = [&](int64_t keys) { return keys > 0 ? w.run_cost + (keys + kTileKeys - 1) / kTileKeys : 0; };
    const int64_t prefix = of(w.n) * w.row_tiles, own = of(w.capacity) * w.batch;
    return (prefix + own) > INT32_MAX / w.heads ? int64_t{INT32_MAX} + 1 : (prefix + own) * w.heads;
}

// workspace of a call: fills the pointers of w from `base` and returns the bytes
// (base may be null: bytes only).  All but base, n, lengths and capacity are set.
int64_t lay_out(Work &w, void *base);

}  // namespace shared

struct SharedArgs {
    const void *q;
    int qdtype;
    const uint8_t *prefix_idx;
    const float *prefix_norms;
    const void *prefix_V;
    int64_t n;
    const uint8_t *idx;
    const float *norms;
    const void *V;
    int64_t capacity;
    const int32_t *lengths;
    int vdtype;
    int batch, heads, group, d, b;
    const int8_t *signs;
    void *workspace;
    void *out;                 // (batch*heads*group, d), vdtype
    float *lse;                // (batch*heads*group), or null
    Codebook cb;
};

// shared_attention.cu: the CUDA-core kernel, the kernel before (rotation, starts)
// and the one after (merge) for both kernels
cudaError_t launch_shared_before(const SharedArgs &a, const shared::Work &w, bool halves, cudaStream_t stream);
cudaError_t launch_shared_after(const SharedArgs &a, const shared::Work &w, cudaStream_t stream);
int64_t shared_workspace_bytes(int batch, int heads, int group, int d);
// whether the line of a call's work has fewer than 2^31 places
bool shared_fits(const SharedArgs &a);
// tensor-core kernel (shared_attention_tc.cu): 16-bit values, d = 64 and 128
bool shared_tc_supported(const SharedArgs &a);
shared::Work shared_tc_work(int batch, int heads, int group, int d);
cudaError_t launch_shared_main_tc(const SharedArgs &a, const shared::Work &w, cudaStream_t stream);
unsigned int shared_tc_status(bool clear);
cudaError_t launch_shared_attention(const SharedArgs &a, cudaStream_t stream);

}  // namespace axr
