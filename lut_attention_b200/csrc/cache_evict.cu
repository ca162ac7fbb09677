// Keeping a cache at a size by accumulated attention weight: the weights of a
// decode step added up per cached key (axr_accumulate_weights), and the choice
// and copy of the rows that stay (axr_evict).
//
// Accumulation: for KV head h and its G queries g,
//     w[h, t] += sum_g e^(s_g[t] - m_g) / l_g,   m_g = max_t s_g[t],  l_g = sum_t e^(s_g[t] - m_g).
// A cluster of kCluster CTAs takes a head and cuts its keys into one stretch per
// CTA: one pass for the running (m, l) of every query, an exchange of the
// kCluster partial (m, l) through distributed shared memory, and a second pass
// that adds the weights (its scores come from L2).  4 G bytes per key are read
// twice and 8 bytes of w moved once.
//
// Eviction of head h with len rows, of which the last `recent` stay anyway:
// among t < len - recent the k = keep - recent rows of largest weight stay,
// equal weights by lowest t.  The weights become unsigned keys in the same order
// and a radix search, 8 bits a round, finds the k-th largest: the head's cluster
// counts its keys per digit in shared memory, the counts meet through distributed
// shared memory, and the digit holding rank k is fixed.  Then one ordered pass
// writes the slots that stay (all above the k-th key, and the first of those
// equal to it), and a second kernel copies the rows.
#include <cooperative_groups.h>

#include "axr_internal.cuh"

namespace axr {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// [begin, end) of CTA `rank`'s stretch of `count` elements
__device__ __forceinline__ void stretch(int count, int rank, int &begin, int &end)
{
    begin = static_cast<int>(static_cast<int64_t>(count) * rank / kCluster);
    end = static_cast<int>(static_cast<int64_t>(count) * (rank + 1) / kCluster);
}

struct WeightParams {
    const float *scores;               // (heads*group, n)
    float *weights;                    // (heads, capacity)
    const int32_t *lengths;            // (heads), or null: n
    int n, capacity, group;
    AXR_DEBUG_ONLY(dbg::Span sp_scores, sp_weights, sp_lengths;)
};

__device__ __forceinline__ int used_rows(const int32_t *lengths, int h, int most AXR_DEBUG_ONLY(, const dbg::Span &sp))
{
    if (!lengths) return most;
    const int len = AXR_IN(sp, lengths + h, 4) ? lengths[h] : 0;
    return min(max(len, 0), most);
}

// (m, l) of two disjoint runs of keys; a NaN score makes l NaN
__device__ __forceinline__ void join(float &m, float &l, float m2, float l2)
{
    const float top = fmaxf(m, m2);
    const float base = top == -INFINITY ? 0.0f : top;
    l = l * expf(m - base) + l2 * expf(m2 - base);
    m = top;
}

template <int G>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) weights_kernel(const WeightParams p)
{
    __shared__ float s_m[kWarps][G], s_l[kWarps][G];
    __shared__ float c_m[G], c_l[G];                          // this CTA's, read by the cluster
    const cg::cluster_group cluster = cg::this_cluster();
    const int h = blockIdx.x / kCluster, rank = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = used_rows(p.lengths, h, p.n AXR_DEBUG_ONLY(, p.sp_lengths));
    int t0, t1;
    stretch(len, rank, t0, t1);
    const float *src = p.scores + static_cast<int64_t>(h) * p.group * p.n;

    float m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.0f;
    }
    constexpr int U = 4;
    for (int t = t0 + threadIdx.x; t < t1; t += U * kThreads) {
        float v[U][G];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float *at = src + static_cast<int64_t>(g) * p.n + t + u * kThreads;
                v[u][g] = (g < p.group && t + u * kThreads < t1 && AXR_IN(p.sp_scores, at, 4)) ? *at : -INFINITY;
            }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float top = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, v[u][g]);
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = l[g] * expf(m[g] - base);
#pragma unroll
            for (int u = 0; u < U; ++u) sum += expf(v[u][g] - base);
            l[g] = sum;
            m[g] = top;
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            join(m[g], l[g], __shfl_xor_sync(0xffffffffu, m[g], o), __shfl_xor_sync(0xffffffffu, l[g], o));
        if (lane == 0) {
            s_m[warp][g] = m[g];
            s_l[warp][g] = l[g];
        }
    }
    __syncthreads();
    if (threadIdx.x < G) {
        float cm = -INFINITY, cl = 0.0f;
        for (int w = 0; w < kWarps; ++w) join(cm, cl, s_m[w][threadIdx.x], s_l[w][threadIdx.x]);
        c_m[threadIdx.x] = cm;
        c_l[threadIdx.x] = cl;
    }
    cluster.sync();
    float base[G], inv[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float cm = -INFINITY, cl = 0.0f;
        for (int r = 0; r < kCluster; ++r) join(cm, cl, *cluster.map_shared_rank(&c_m[g], r), *cluster.map_shared_rank(&c_l[g], r));
        base[g] = cm == -INFINITY ? 0.0f : cm;
        inv[g] = cl > 0.0f ? 1.0f / cl : cl;                  // a query without a key adds nothing, NaN stays NaN
    }
    cluster.sync();                                           // no CTA leaves while its (m, l) are read
    float *dst = p.weights + static_cast<int64_t>(h) * p.capacity;
    for (int t = t0 + threadIdx.x; t < t1; t += kThreads) {
        if (!AXR_IN(p.sp_weights, dst + t, 4)) continue;
        float w = dst[t];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float *at = src + static_cast<int64_t>(g) * p.n + t;
            if (g < p.group && AXR_IN(p.sp_scores, at, 4)) w = fmaf(expf(*at - base[g]), inv[g], w);
        }
        dst[t] = w;
    }
}

struct EvictParams {
    const float *weights;              // (heads, capacity)
    const int32_t *lengths;            // (heads)
    int capacity, keep, recent;
    int *kept;                         // (heads, keep)
    int32_t *lengths_out;              // (heads)
    AXR_DEBUG_ONLY(dbg::Span sp_weights, sp_lengths, sp_kept, sp_lengths_out;)
};

// order-preserving: larger weight, larger key; -0 equals +0; NaN below all
__device__ __forceinline__ uint32_t key_of(float w)
{
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);             // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) choose_kernel(const EvictParams p)
{
    __shared__ int hist[256];                                 // read by the cluster
    __shared__ int total[256];
    __shared__ int s_above, s_equal;                          // this CTA's counts, read by the cluster
    __shared__ int s_digit, s_rank;
    __shared__ int warp_above[kWarps], warp_equal[kWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const int h = blockIdx.x / kCluster, rank = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = used_rows(p.lengths, h, p.capacity AXR_DEBUG_ONLY(, p.sp_lengths));
    int *kept = p.kept + static_cast<int64_t>(h) * p.keep;
    auto put = [&](int at, int t) {
        if (AXR_IN(p.sp_kept, kept + at, 4)) kept[at] = t;
    };
    if (rank == 0 && threadIdx.x == 0 && AXR_IN(p.sp_lengths_out, p.lengths_out + h, 4))
        p.lengths_out[h] = min(len, p.keep);
    if (len <= p.keep) {                                      // the whole cluster: all rows stay
        for (int i = rank * kThreads + threadIdx.x; i < p.keep; i += kCluster * kThreads) put(i, i < len ? i : -1);
        return;
    }
    const int old = len - p.recent, k = p.keep - p.recent;    // k of the first `old` rows stay, k < old
    for (int i = rank * kThreads + threadIdx.x; i < p.recent; i += kCluster * kThreads) put(k + i, old + i);
    if (k == 0) return;                                       // the whole cluster
    int t0, t1;
    stretch(old, rank, t0, t1);
    const float *src = p.weights + static_cast<int64_t>(h) * p.capacity;
    auto key_at = [&](int t) { return AXR_IN(p.sp_weights, src + t, 4) ? key_of(__ldg(src + t)) : 0u; };

    uint32_t prefix = 0;                                      // the digits fixed so far
    int want = k;                                             // rank of the k-th largest among keys with that prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int t = t0 + threadIdx.x; t < t1; t += kThreads) {
            const uint32_t key = key_at(t);
            if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        cluster.sync();
        if (threadIdx.x < 256) {
            int sum = 0;
            for (int r = 0; r < kCluster; ++r) sum += cluster.map_shared_rank(hist, r)[threadIdx.x];
            total[threadIdx.x] = sum;
        }
        cluster.sync();                                       // total is whole; no CTA clears counts that are read
        if (warp == 0) {                                      // the digit where the count from above reaches `want`
            int own[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                own[i] = total[255 - (lane * 8 + i)];
                sum += own[i];
            }
            int upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            int before = upto - sum;
            if (before < want && want <= upto) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < want && want <= before + own[i]) {
                        s_digit = 255 - (lane * 8 + i);
                        s_rank = want - before;
                    }
                    before += own[i];
                }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(s_digit);
        want = s_rank;
        __syncthreads();
    }
    // keys above `prefix` stay, and of those equal to it the first `want`
    int above = 0, equal = 0;
    for (int t = t0 + threadIdx.x; t < t1; t += kThreads) {
        const uint32_t key = key_at(t);
        above += key > prefix;
        equal += key == prefix;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        warp_above[warp] = above;
        warp_equal[warp] = equal;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int a = 0, e = 0;
        for (int i = 0; i < kWarps; ++i) {
            a += warp_above[i];
            e += warp_equal[i];
        }
        s_above = a;
        s_equal = e;
    }
    cluster.sync();
    int above_before = 0, equal_before = 0;
    for (int r = 0; r < rank; ++r) {
        above_before += *cluster.map_shared_rank(&s_above, r);
        equal_before += *cluster.map_shared_rank(&s_equal, r);
    }
    cluster.sync();                                           // no CTA leaves while its counts are read
    for (int base = t0; base < t1; base += kThreads) {        // in order, kThreads rows at a time
        const int t = base + threadIdx.x;
        const uint32_t key = t < t1 ? key_at(t) : 0u;
        const bool is_above = t < t1 && key > prefix, is_equal = t < t1 && key == prefix;
        const unsigned ba = __ballot_sync(0xffffffffu, is_above), be = __ballot_sync(0xffffffffu, is_equal);
        if (lane == 0) {
            warp_above[warp] = __popc(ba);
            warp_equal[warp] = __popc(be);
        }
        __syncthreads();
        int a = above_before, e = equal_before, all_a = above_before, all_e = equal_before;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) {
                a += warp_above[i];
                e += warp_equal[i];
            }
            all_a += warp_above[i];
            all_e += warp_equal[i];
        }
        const unsigned lower = (1u << lane) - 1u;
        a += __popc(ba & lower);
        e += __popc(be & lower);
        if (is_above || (is_equal && e < want)) put(a + min(e, want), t);
        above_before = all_a;
        equal_before = all_e;
        __syncthreads();
    }
}

struct CopyParams {
    const int *kept;                   // (heads, keep), -1: none
    int keep;
    int capacity, capacity_out;
    const char *idx, *V;
    char *idx_out, *V_out;
    const float *norms, *weights;
    float *norms_out, *weights_out;
    int p_bytes, v_bytes;
    AXR_DEBUG_ONLY(dbg::Span sp_kept, sp_idx, sp_V, sp_norms, sp_weights, sp_idx_out, sp_V_out, sp_norms_out, sp_weights_out;)
};

constexpr int kCopyRows = 32;          // rows of a CTA
constexpr int kCopyThreads = 256;

// CTA: kCopyRows rows of one head; a value row is v_bytes / 16 pieces, a packed
// row p_bytes / sizeof(U) pieces
template <typename U>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyParams p)
{
    __shared__ int s_from[kCopyRows];
    const int h = blockIdx.y, i0 = blockIdx.x * kCopyRows;
    const int rows = min(kCopyRows, p.keep - i0);
    const int64_t from0 = static_cast<int64_t>(h) * p.capacity, to0 = static_cast<int64_t>(h) * p.capacity_out + i0;
    if (threadIdx.x < rows) {
        const int *src = p.kept + static_cast<int64_t>(h) * p.keep + i0 + threadIdx.x;
        const int t = AXR_IN(p.sp_kept, src, 4) ? *src : -1;
        s_from[threadIdx.x] = t;
        if (t >= 0) {
            const float *n = p.norms + from0 + t, *w = p.weights + from0 + t;
            float *no = p.norms_out + to0 + threadIdx.x, *wo = p.weights_out + to0 + threadIdx.x;
            if (AXR_IN(p.sp_norms, n, 4) && AXR_IN(p.sp_norms_out, no, 4)) *no = *n;
            if (AXR_IN(p.sp_weights, w, 4) && AXR_IN(p.sp_weights_out, wo, 4)) *wo = *w;
        }
    }
    __syncthreads();
    const int vp = p.v_bytes / 16;
    for (int c = threadIdx.x; c < rows * vp; c += kCopyThreads) {
        const int i = c / vp, e = c % vp;
        if (s_from[i] < 0) continue;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.V + (from0 + s_from[i]) * p.v_bytes) + e;
        uint4 *dst = reinterpret_cast<uint4 *>(p.V_out + (to0 + i) * p.v_bytes) + e;
        if (AXR_IN(p.sp_V, src, 16) && AXR_IN(p.sp_V_out, dst, 16)) *dst = __ldcs(src);
    }
    const int pp = p.p_bytes / static_cast<int>(sizeof(U));
    for (int c = threadIdx.x; c < rows * pp; c += kCopyThreads) {
        const int i = c / pp, e = c % pp;
        if (s_from[i] < 0) continue;
        const U *src = reinterpret_cast<const U *>(p.idx + (from0 + s_from[i]) * p.p_bytes) + e;
        U *dst = reinterpret_cast<U *>(p.idx_out + (to0 + i) * p.p_bytes) + e;
        if (AXR_IN(p.sp_idx, src, sizeof(U)) && AXR_IN(p.sp_idx_out, dst, sizeof(U))) *dst = __ldcs(src);
    }
}

}  // namespace

cudaError_t launch_accumulate_weights(const WeightArgs &a, cudaStream_t stream)
{
    WeightParams p{};
    p.scores = a.scores;
    p.weights = a.weights;
    p.lengths = a.lengths;
    p.n = static_cast<int>(a.n);
    p.capacity = static_cast<int>(a.capacity);
    p.group = a.group;
    AXR_DEBUG_ONLY(p.sp_scores = dbg::span(a.scores, 4ull * a.heads * a.group * a.n);
                   p.sp_weights = dbg::span(a.weights, 4ull * a.heads * a.capacity);
                   p.sp_lengths = dbg::span(a.lengths, a.lengths ? 4ull * a.heads : 0);)
    const unsigned grid = static_cast<unsigned>(a.heads) * kCluster;
    if (a.group <= 1) weights_kernel<1><<<grid, kThreads, 0, stream>>>(p);
    else if (a.group <= 2) weights_kernel<2><<<grid, kThreads, 0, stream>>>(p);
    else if (a.group <= 4) weights_kernel<4><<<grid, kThreads, 0, stream>>>(p);
    else weights_kernel<8><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t stream)
{
    EvictParams p{};
    p.weights = a.weights;
    p.lengths = a.lengths;
    p.capacity = static_cast<int>(a.capacity);
    p.keep = static_cast<int>(a.keep);
    p.recent = static_cast<int>(a.recent);
    p.kept = a.kept;
    p.lengths_out = a.lengths_out;
    AXR_DEBUG_ONLY(p.sp_weights = dbg::span(a.weights, 4ull * a.heads * a.capacity);
                   p.sp_lengths = dbg::span(a.lengths, 4ull * a.heads);
                   p.sp_kept = dbg::span(a.kept, 4ull * a.heads * a.keep);
                   p.sp_lengths_out = dbg::span(a.lengths_out, 4ull * a.heads);)
    choose_kernel<<<static_cast<unsigned>(a.heads) * kCluster, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    CopyParams c{};
    c.kept = a.kept;
    c.keep = p.keep;
    c.capacity = p.capacity;
    c.capacity_out = static_cast<int>(a.capacity_out);
    c.idx = reinterpret_cast<const char *>(a.idx);
    c.V = static_cast<const char *>(a.V);
    c.idx_out = reinterpret_cast<char *>(a.idx_out);
    c.V_out = static_cast<char *>(a.V_out);
    c.norms = a.norms;
    c.weights = a.weights;
    c.norms_out = a.norms_out;
    c.weights_out = a.weights_out;
    c.p_bytes = a.d * a.b / 8;
    c.v_bytes = a.d * dtype_bytes(a.vdtype);
    AXR_DEBUG_ONLY(const uint64_t rows = static_cast<uint64_t>(a.heads) * a.capacity;
                   const uint64_t rows_out = static_cast<uint64_t>(a.heads) * a.capacity_out;
                   c.sp_kept = p.sp_kept; c.sp_weights = p.sp_weights;
                   c.sp_idx = dbg::span(a.idx, rows * c.p_bytes); c.sp_V = dbg::span(a.V, rows * c.v_bytes);
                   c.sp_norms = dbg::span(a.norms, rows * 4);
                   c.sp_idx_out = dbg::span(a.idx_out, rows_out * c.p_bytes);
                   c.sp_V_out = dbg::span(a.V_out, rows_out * c.v_bytes);
                   c.sp_norms_out = dbg::span(a.norms_out, rows_out * 4);
                   c.sp_weights_out = dbg::span(a.weights_out, rows_out * 4);)
    const dim3 grid((p.keep + kCopyRows - 1) / kCopyRows, a.heads);
    if (c.p_bytes % 16 == 0) copy_kernel<uint4><<<grid, kCopyThreads, 0, stream>>>(c);
    else if (c.p_bytes % 4 == 0) copy_kernel<uint32_t><<<grid, kCopyThreads, 0, stream>>>(c);
    else copy_kernel<uint8_t><<<grid, kCopyThreads, 0, stream>>>(c);
    return cudaGetLastError();
}

}  // namespace axr
