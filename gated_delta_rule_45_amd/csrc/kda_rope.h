// Rotation of 16 channels of a head by position-dependent angles, shared by the rotary kernel and by the one
// that appends to the cache.
#pragma once

#include "kda_device.h"

namespace kda {
namespace paged {

// cos and sin of position * f.  The product is taken in 64 bits, in quarter turns: at position 2^20 a 32-bit angle
// would be off by up to 2^-5.  What is left of a quarter turn, at most pi / 4, is exact to 2^-53 of the angle and
// goes into the power series (the first terms left out are 2e-9 and 2e-9 of 1).
__device__ __forceinline__ void angle(int pos, float f, float &c, float &s) {
    const double q = (double)pos * (double)f * 0.63661977236758134308;  // 2 / pi
    const double n = rint(q);
    const float x = (float)((q - n) * 1.57079632679489661923);
    const int quarter = (int)(n - 4.0 * floor(0.25 * n));
    const float z = x * x;
    const float sx = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float cx = fmaf(
        z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    const float a = quarter & 1 ? sx : cx, b = quarter & 1 ? cx : sx;
    c = (quarter == 1 || quarter == 2) ? -a : a;
    s = quarter >= 2 ? -b : b;
}

// 8 consecutive values of a row as they lie in memory, and as fp32.
template <typename IO>
struct Eight {
    static constexpr int W = sizeof(IO) / 2;  // 16-byte words
    u32x4 w[W];
    __device__ __forceinline__ void load(const IO *p) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const u32x4 *>(p)[i];
    }
    __device__ __forceinline__ void store(IO *p) const {
#pragma unroll
        for (int i = 0; i < W; ++i) reinterpret_cast<u32x4 *>(p)[i] = w[i];
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (W == 1) {
            return i & 1 ? bf16_hi(w[0][i / 2]) : bf16_lo(w[0][i / 2]);
        } else {
            return __uint_as_float(w[i / 4][i % 4]);
        }
    }
    __device__ __forceinline__ void put2(int i, float a, float b) {  // i even
        if constexpr (W == 1) {
            w[0][i / 2] = pack_bf16x2(a, b);
        } else {
            w[i / 4][i % 4] = __float_as_uint(a);
            w[i / 4][i % 4 + 1] = __float_as_uint(b);
        }
    }
};

// Unit u of a head: 8 pairs.  Halves: channels 8 u .. and rot / 2 + 8 u ..; neighbours: 16 u .. 16 u + 15.  Both move
// as two runs of 8.
struct Turn {
    float c[8], s[8];
    __device__ __forceinline__ void set(int pos, const float *freq, int u, float amplitude, float sign) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            angle(pos, freq[8 * u + i], c[i], s[i]);
            c[i] *= amplitude;
            s[i] *= amplitude * sign;
        }
    }
    template <typename IO>
    __device__ __forceinline__ void apply(Eight<IO> &a, Eight<IO> &b, int interleaved) const {
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = a.get(2 * i), y = a.get(2 * i + 1), z = b.get(2 * i), w = b.get(2 * i + 1);
                a.put2(2 * i, fmaf(x, c[i], -y * s[i]), fmaf(x, s[i], y * c[i]));
                b.put2(2 * i, fmaf(z, c[4 + i], -w * s[4 + i]), fmaf(z, s[4 + i], w * c[4 + i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float x0 = a.get(i), x1 = a.get(i + 1), y0 = b.get(i), y1 = b.get(i + 1);
                a.put2(i, fmaf(x0, c[i], -y0 * s[i]), fmaf(x1, c[i + 1], -y1 * s[i + 1]));
                b.put2(i, fmaf(x0, s[i], y0 * c[i]), fmaf(x1, s[i + 1], y1 * c[i + 1]));
            }
        }
    }
};

// Where the two runs of unit u start: turned units come first, copied ones (16 channels as they are) behind them.
__device__ __forceinline__ int run0(int u, int rot, int interleaved) { return 16 * u < rot && !interleaved ? 8 * u : 16 * u; }
__device__ __forceinline__ int run1(int u, int rot, int interleaved) {
    return 16 * u < rot && !interleaved ? rot / 2 + 8 * u : 16 * u + 8;
}

}  // namespace paged
}  // namespace kda
