// block8.h -- from values to e4m3 with a power-of-two scale for a block of 128:
// the largest magnitude, the scale's byte and the conversion (fp8.hip, rms.hip).
#pragma once

#include "engram_internal.h"
#include "vec8.h"

namespace engram {

// Largest magnitudes of 8 columns as bit patterns (which order like the
// values), two bf16 columns a word.  NaN and infinity are above kNotFinite.
constexpr uint32_t kNotFinite = 0x7F800000u;
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                  __builtin_bit_cast(u16x2_t, b)));
}

template <typename T>
struct Top8;
template <>
struct Top8<uint16_t> {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    __device__ __forceinline__ void add(const Raw8<uint16_t> &x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = max_u16x2(w[i], x.w[i] & 0x7FFF7FFFu);
    }
    __device__ __forceinline__ uint32_t column(int i) const { return (i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16; }
    __device__ __forceinline__ uint32_t all() const {
        const uint32_t m = max_u16x2(max_u16x2(w[0], w[1]), max_u16x2(w[2], w[3]));
        return max(m & 0xFFFF0000u, m << 16);
    }
};
template <>
struct Top8<float> {
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    __device__ __forceinline__ void add(const Raw8<float> &x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = max(w[i], __float_as_uint(x.a[i]) & 0x7FFFFFFFu);
            w[4 + i] = max(w[4 + i], __float_as_uint(x.b[i]) & 0x7FFFFFFFu);
        }
    }
    __device__ __forceinline__ uint32_t column(int i) const { return w[i]; }
    __device__ __forceinline__ uint32_t all() const {
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, w[i]);
        return m;
    }
};

// |x| as bits, 0 where x is not finite
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
    return b < kNotFinite ? b : 0u;
}

// Biased exponent of the block's scale from the bits of its largest finite
// magnitude (448 = 1.75 * 2^8).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(e, 1);
}

// 1 / scale: exact (a power of two in the normal range, 2^-120 .. 2^126)
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// To e4m3 bytes.  Finite values are at most 448 here; the conversion makes NaN
// of infinities, which e4m3 does not have.
__device__ __forceinline__ u32x2_t cvt8(const F8 &x, float inv) {
    u32x2_t q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(x.v[4 * i] * inv, x.v[4 * i + 1] * inv, 0, false);
        q[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x.v[4 * i + 2] * inv, x.v[4 * i + 3] * inv, w, true);
    }
    return q;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}
// over the 16 lanes of a row (neighbours, quads, halves, the row's mirror)
__device__ __forceinline__ uint32_t max16(uint32_t x) { return dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(x)))); }

}  // namespace engram
