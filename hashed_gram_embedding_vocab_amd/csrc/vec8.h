// vec8.h -- eight consecutive bf16 or fp32 elements moved as fp32 values: the
// unit in which the row kernels (embed.hip, norm.hip, fp8.hip) read and write.
// Rounding to bf16 is to nearest even and keeps NaN and infinity.
#pragma once

#include "engram_internal.h"

namespace engram {

// x / d for x >= 0, in 32 bits where x fits (a 64-bit division is a few hundred
// instructions, which a short kernel's waves would start with).
__device__ __forceinline__ int64_t quotient(int64_t x, int32_t d) {
    return (x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : x / d;
}

// 8 consecutive elements as fp32, from 16 bytes of bf16 or 32 of fp32
struct F8 {
    float v[8];
};

// The same unit as loaded: half the registers for bf16 while a load is in flight.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4_t w;
    __device__ __forceinline__ F8 get() const {
        F8 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[2 * i] = __uint_as_float(w[i] << 16);
            r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        return r;
    }
};
template <>
struct Raw8<float> {
    f32x4_t a, b;
    __device__ __forceinline__ F8 get() const { return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}}; }
};
__device__ __forceinline__ Raw8<uint16_t> load_raw8(const uint16_t *p) {
    return Raw8<uint16_t>{*reinterpret_cast<const u32x4_t *>(p)};
}
__device__ __forceinline__ Raw8<float> load_raw8(const float *p) {
    return Raw8<float>{*reinterpret_cast<const f32x4_t *>(p), *reinterpret_cast<const f32x4_t *>(p + 4)};
}
template <typename T>
__device__ __forceinline__ F8 load8(const T *p) {
    return load_raw8(p).get();
}
__device__ __forceinline__ void store8(uint16_t *p, const F8 &x) {
    *reinterpret_cast<u32x4_t *>(p) = u32x4_t{pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]),
                                              pack_bf16x2(x.v[4], x.v[5]), pack_bf16x2(x.v[6], x.v[7])};
}
__device__ __forceinline__ void store8(float *p, const F8 &x) {
    *reinterpret_cast<f32x4_t *>(p) = f32x4_t{x.v[0], x.v[1], x.v[2], x.v[3]};
    *reinterpret_cast<f32x4_t *>(p + 4) = f32x4_t{x.v[4], x.v[5], x.v[6], x.v[7]};
}

}  // namespace engram
