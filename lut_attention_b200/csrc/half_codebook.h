// The codebook in fp16 for the tensor cores (host): centroid i is held as
// fp16(scale * c_i).  Any power of two may be folded into the scores afterwards,
// and so may any other scale: one is searched for which all of the at most eight
// magnitudes c_i land close to fp16 numbers.  A random scale rounds each by up to
// 2^-11 relatively; the best of 2^16 candidates in [1, 2) keeps all eight within 2^-13.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

namespace axr {

struct HalfCodebook {
    uint16_t bits[16];         // fp16 of scale * c_i
    float scale;
    float worst;               // largest relative rounding error
};

// nearest fp16 number of a positive value well inside fp16's normal range (ties to even)
inline double nearest_half(double v, uint16_t *bits)
{
    int e = 0;
    const double f = std::frexp(v, &e);                        // v = f 2^e, f in [1/2, 1)
    double m = std::nearbyint(f * 2048.0);                     // 11 bits
    if (m == 2048.0) {
        m = 1024.0;
        ++e;
    }
    if (bits) *bits = static_cast<uint16_t>(((e + 14) << 10) + (static_cast<int>(m) - 1024));
    return std::ldexp(m, e - 11);
}

inline HalfCodebook half_codebook(const float *centroids, int d, int b)
{
    const int L = 1 << b, m = L / 2;
    const double unit = std::sqrt(static_cast<double>(d));     // brings the centroids near 1
    constexpr int kTries = 1 << 16;
    double best = 1.0, best_scale = 1.0;
    for (int k = 0; k < kTries; ++k) {
        const float s = static_cast<float>(unit * (1.0 + static_cast<double>(k) / kTries));
        double worst = 0.0;
        for (int i = m; i < L && worst < best; ++i) {
            const double v = static_cast<double>(s) * centroids[i];
            worst = std::fmax(worst, std::fabs(nearest_half(v, nullptr) - v) / v);
        }
        if (worst < best) {
            best = worst;
            best_scale = s;
        }
    }
    HalfCodebook out;
    std::memset(&out, 0, sizeof(out));
    out.scale = static_cast<float>(best_scale);
    out.worst = static_cast<float>(best);
    for (int i = m; i < L; ++i) {
        nearest_half(best_scale * centroids[i], &out.bits[i]);
        out.bits[L - 1 - i] = static_cast<uint16_t>(out.bits[i] | 0x8000u);
    }
    return out;
}

}  // namespace axr
