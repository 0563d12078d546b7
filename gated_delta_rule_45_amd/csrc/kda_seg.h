// One 16-byte segment of a row of io values as fp32 (output epilogue and its gradients).
#pragma once

#include "kda_device.h"

namespace kda {

template <typename IO>
struct Seg;  // one 16-byte segment of a row as fp32 values
template <>
struct Seg<uint16_t> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void load(const uint16_t *p, float (&v)[N]) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    __device__ static __forceinline__ void store(uint16_t *p, const float (&v)[N]) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<u32x4 *>(p) = w;
    }
};
template <>
struct Seg<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void load(const float *p, float (&v)[N]) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w[i];
    }
    __device__ static __forceinline__ void store(float *p, const float (&v)[N]) {
        f32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v[i];
        *reinterpret_cast<f32x4 *>(p) = w;
    }
};

}  // namespace kda
