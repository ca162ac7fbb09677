// Softmax arithmetic of the tensor-core attention kernels: one thread holds a
// query's scores of a tile in registers and turns them into 16-bit weights.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace axr {
namespace softmax {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 of the growth of a query's maximum that rescales its sums
constexpr float kLazy = 8.0f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// two weights as packed 16-bit values, the first in the low half
template <bool kBF16>
__device__ __forceinline__ uint32_t pack16(float a, float b)
{
    uint32_t r;
    if constexpr (kBF16) asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    else asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    return r;
}

// fp16 weights carry a factor 2^7: with the lazy maximum they reach 2^15 at most,
// and those as small as 2^-21 of the largest are still normal numbers
template <bool kBF16>
constexpr float kBias = kBF16 ? 0.0f : 7.0f;

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The tile loops below are rolled into chunks of 32 columns on purpose: unrolled
// over a tile their code is streamed through the instruction caches once a tile,
// and every other role of the SM waits for instructions.

// largest of 32 scores and `m`
__device__ __forceinline__ float max32(const uint32_t (&s)[32], float m)
{
    float top[2] = {m, __uint_as_float(s[0])};
#pragma unroll
    for (int i = 1; i < 29; i += 4) {
        top[0] = max3(top[0], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        top[1] = max3(top[1], __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
    }
    top[0] = max3(top[0], __uint_as_float(s[29]), __uint_as_float(s[30]));
    return max3(top[0], top[1], __uint_as_float(s[31]));
}

// scores from column `lim` on to -inf
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int lim)
{
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (c >= lim) s[c] = 0xff800000u;
}

// Softmax of 32 scores: p = 2^(s * scale + c), their sum into (sum0, sum1), packed into w
template <bool kBF16>
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], uint64_t scale2, uint64_t c2, uint64_t &sum0,
                                          uint64_t &sum1, uint32_t (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float a, b;
        unpair(fma2(pair(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), scale2, c2), a, b);
        a = ex2(a);
        b = ex2(b);
        if (i & 2) sum1 = add2(sum1, pair(a, b));
        else sum0 = add2(sum0, pair(a, b));
        w[i / 2] = pack16<kBF16>(a, b);
    }
}

}  // namespace softmax
}  // namespace axr
