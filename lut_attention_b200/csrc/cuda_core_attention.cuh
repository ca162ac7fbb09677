// One block of softmax attention on the CUDA cores, in fp32: the queries of a
// tile against successive tiles of keys and values, one pass over the keys with
// the running maximum m and sum l of each query's softmax,
//     m' = max(m, max_t s_t),  a = 2^(m - m'),
//     l  <- a l + sum_t 2^(s_t - m'),  o <- a o + sum_t 2^(s_t - m') V_t,
// with s in units of log2 (the queries carry the factor log2 e).  Serves fp32
// operands and the head widths the tensor-core kernels do not take.
//
// 256 threads as 16 x 16: thread (ty, tx) owns queries ty + 16 i and, of the
// scores, keys tx + 16 j; of the output, D / 16 coordinates.  The 16 threads of
// a query sit in one half-warp, so its statistics are shuffles and its weights
// pass through shared memory behind a __syncwarp.  Rows are padded by 16 bytes,
// which keeps the 16-byte reads of neighbouring rows free of bank conflicts.  Both
// products are bound by the FMA pipes and run on pairs of fp32 numbers, which leaves
// issue slots to the shared-memory reads: even and odd coordinates of a score in the
// two halves, neighbouring coordinates of an output.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "packed_f32.cuh"

namespace axr {
namespace core {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v)
{
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// keys per tile and padded row strides (floats)
template <int D>
struct Shape {
    static constexpr int BN = D <= 128 ? 64 : 32;
    static constexpr int DS = D + 4;
    static constexpr int PS = BN + 4;
    static constexpr int E = D / 16;             // output coordinates per thread
    static constexpr int W = E < 4 ? E : 4;      // of which consecutive
};

// shared memory of a tile of BM queries (floats)
template <int D, int BM>
constexpr int smem_floats()
{
    using S = Shape<D>;
    return BM * S::DS + 2 * S::BN * S::DS + BM * S::PS;
}

template <int D, int BM>
struct Tile {
    using S = Shape<D>;
    static constexpr int R = BM / 16, C = S::BN / 16, E = S::E, W = S::W;
    float *q, *k, *v, *p;                        // q [BM][DS], k and v [BN][DS], p [BM][PS]
    float m[R], l[R];
    uint64_t o[R][E / 2];                        // pairs of coordinates

    __device__ explicit Tile(float *smem)
        : q(smem), k(q + BM * S::DS), v(k + S::BN * S::DS), p(v + S::BN * S::DS)
    {
    }
    __device__ void reset()
    {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) o[i][e] = 0u;     // two zeros
        }
    }
    __device__ int ty() const { return threadIdx.x >> 4; }
    __device__ int tx() const { return threadIdx.x & 15; }
    __device__ int row(int i) const { return ty() + 16 * i; }
    // output e of query row(i)
    __device__ float out(int i, int e) const
    {
        float a, b;
        packed::unpair(o[i][e / 2], a, b);
        return e & 1 ? b : a;
    }
    // output coordinate e of this thread
    __device__ int col(int e) const { return (e / W) * 16 * W + tx() * W + e % W; }

    // One tile of keys in k and v (valid after a __syncthreads): limit(row) is
    // the number of the tile's keys that query row sees (0 or less: none).
    template <typename Limit>
    __device__ void step(Limit limit)
    {
        using namespace packed;
        float s[R][C];
        {
            uint64_t s2[R][C];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < C; ++j) s2[i][j] = 0u;    // two zeros
#pragma unroll 2
            for (int x = 0; x < D; x += 4) {
                ulonglong2 a[R], b[C];
#pragma unroll
                for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const ulonglong2 *>(q + row(i) * S::DS + x);
#pragma unroll
                for (int j = 0; j < C; ++j) b[j] = *reinterpret_cast<const ulonglong2 *>(k + (tx() + 16 * j) * S::DS + x);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < C; ++j) s2[i][j] = fma2(a[i].y, b[j].y, fma2(a[i].x, b[j].x, s2[i][j]));
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    float even, odd;
                    unpair(s2[i][j], even, odd);
                    s[i][j] = even + odd;
                }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int lim = limit(row(i));
            float top = m[i];
#pragma unroll
            for (int j = 0; j < C; ++j) {
                if (tx() + 16 * j >= lim) s[i][j] = -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            // a query that has seen no key yet keeps weights of 0
            const float base = top == -INFINITY ? 0.0f : top;
            const float a = exp2f(m[i] - base);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float w = exp2f(s[i][j] - base);
                sum += w;
                p[row(i) * S::PS + tx() + 16 * j] = w;
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l[i] = fmaf(l[i], a, sum);
            m[i] = top;
            const uint64_t a2 = pair(a, a);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) o[i][e] = mul2(o[i][e], a2);
        }
        __syncwarp();
        for (int t = 0; t < S::BN; t += 4) {
            float4 w[R];
#pragma unroll
            for (int i = 0; i < R; ++i) w[i] = *reinterpret_cast<const float4 *>(p + row(i) * S::PS + t);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint64_t x[E / 2];
#pragma unroll
                for (int e = 0; e < E; e += W) {
                    const float *src = v + (t + u) * S::DS + col(e);
                    if constexpr (W == 4) {
                        const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(src);
                        x[e / 2] = y.x;
                        x[e / 2 + 1] = y.y;
                    } else {
                        x[e / 2] = *reinterpret_cast<const uint64_t *>(src);
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float wi = u == 0 ? w[i].x : u == 1 ? w[i].y : u == 2 ? w[i].z : w[i].w;
                    const uint64_t w2 = pair(wi, wi);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) o[i][e] = fma2(w2, x[e], o[i][e]);
                }
            }
        }
        __syncwarp();
    }
};

}  // namespace core
}  // namespace axr
