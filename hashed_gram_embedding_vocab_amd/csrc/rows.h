// rows.h -- how the norms (norm.hip, rms.hip) spread a row of channels over lanes
// and waves, its sums, and the join of the blocks' parameter gradients.
#pragma once

#include <algorithm>

#include "engram_internal.h"
#include "vec8.h"

namespace engram {
namespace {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

// Sum over the L lanes of a row (all of them get it): neighbours, quads, halves
// of a row of 16 and its mirror by DPP, the four rows of a wave by readlane
// (a shuffle through the LDS crossbar takes several times as long).
template <int L>
__device__ __forceinline__ float lane_sum(float x) {
    x = dpp_add<0xB1>(x);   // lane ^ 1
    x = dpp_add<0x4E>(x);   // lane ^ 2
    x = dpp_add<0x141>(x);  // the other quad of 8
    if constexpr (L >= 16) x = dpp_add<0x140>(x);  // the other 8 of 16
    if constexpr (L == 32) x += __shfl_xor(x, 16);
    if constexpr (L == 64) {
        const int b = __float_as_int(x);
        x = (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
            (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
    }
    return x;
}

// Sums over the lanes and waves of a row.  `turn` alternates between two LDS
// slots, so one barrier a sum is enough: a slot is written again only after
// the barrier of the sum in between.
template <int L, int W, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*red)[2][N][W], int wave, int lane, int &turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane_sum<L>(x[i]);
    if constexpr (W > 1) {
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) (*red)[turn][i][wave] = x[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) x[i] += (*red)[turn][i][j];
        }
        turn ^= 1;
    }
}

// How a kernel's blocks take rows: 256 threads and 4 * 64 / L rows at a time
// where W == 1, else 64 W threads and one row.
template <int L, int W>
struct Rows {
    static constexpr int kAtOnce = W == 1 ? 256 / L : 1;
    int wave, lane, c0, slot;
    __device__ __forceinline__ Rows() {
        lane = threadIdx.x & 63;
        wave = W == 1 ? 0 : threadIdx.x >> 6;
        slot = W == 1 ? (int)threadIdx.x / L : 0;
        c0 = (wave * 64 + lane % L) * 8;  // channels c0 + 512 W j .. + 7
    }
};

// dst[q][i] (+)= the sum over the blocks of part[q][block][i]: 64 channels a
// workgroup, 16 waves each adding every 16th block in order, then the waves in order.
__global__ __launch_bounds__(1024) void norm_bwd_sum_kernel(const float *part, int32_t blocks, int32_t d,
                                                            bool accumulate, float *dgamma, float *dbeta) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int32_t i = (int32_t)blockIdx.x * 64 + lane;
    float *dst = blockIdx.y == 0 ? dgamma : dbeta;
    if (!dst) return;
    const float *p = part + (int64_t)blockIdx.y * blocks * d;
    float acc = 0.f;
    if (i < d) {
#pragma unroll 8
        for (int32_t b = w; b < blocks; b += 16) acc += p[(int64_t)b * d + i];
    }
    red[w][lane] = acc;
    __syncthreads();
    if (w == 0 && i < d) {
        float t = red[0][lane];
#pragma unroll
        for (int j = 1; j < 16; ++j) t += red[j][lane];
        dst[i] = accumulate ? dst[i] + t : t;
    }
}

// How a row is spread: 8 to 32 lanes up to 256 channels, one wave up to 2560
// (five steps; 262 registers in the bf16 backward and 308 in the fp32 one, so
// one wave a SIMD there), then 2 to 16 waves.
struct RowShape {
    int lanes, waves, steps;
    int at_once() const { return waves == 1 ? 256 / lanes : 1; }
};
inline RowShape row_shape(int32_t d) {
    if (d <= 256) return RowShape{d <= 64 ? 8 : d <= 128 ? 16 : 32, 1, 1};
    const int units = (d + 511) / 512;
    int w = 1;
    while (w < 16 && (units + w - 1) / w > (w == 1 ? 5 : 4)) w *= 2;
    return RowShape{64, w, (units + w - 1) / w};
}

// Blocks: per_cu times 4 waves for each of 256 CUs, or one for each where that
// is less.  (Where the registers hold fewer at once, as in the five-step
// backward with one of its two, the others follow.)
inline int64_t norm_blocks(const RowShape &sh, int64_t n_rows, int per_cu) {
    const int64_t waves = sh.waves == 1 ? 4 : sh.waves;
    return std::min<int64_t>((n_rows + sh.at_once() - 1) / sh.at_once(), std::max<int64_t>(256, 256 * per_cu * 4 / waves));
}

#define ENGRAM_NORM_CASE(FN, L, W, N) \
    case (L * 32 + W) * 8 + N: FN(L, W, N); break;
#define ENGRAM_NORM_SWITCH(FN, SHAPE)                                                                     \
    switch (((SHAPE).lanes * 32 + (SHAPE).waves) * 8 + (SHAPE).steps) {                                   \
        ENGRAM_NORM_CASE(FN, 8, 1, 1) ENGRAM_NORM_CASE(FN, 16, 1, 1) ENGRAM_NORM_CASE(FN, 32, 1, 1)       \
        ENGRAM_NORM_CASE(FN, 64, 1, 1) ENGRAM_NORM_CASE(FN, 64, 1, 2) ENGRAM_NORM_CASE(FN, 64, 1, 3)      \
        ENGRAM_NORM_CASE(FN, 64, 1, 4) ENGRAM_NORM_CASE(FN, 64, 1, 5)                                     \
        ENGRAM_NORM_CASE(FN, 64, 2, 3) ENGRAM_NORM_CASE(FN, 64, 2, 4)                                     \
        ENGRAM_NORM_CASE(FN, 64, 4, 3) ENGRAM_NORM_CASE(FN, 64, 4, 4)                                     \
        ENGRAM_NORM_CASE(FN, 64, 8, 3) ENGRAM_NORM_CASE(FN, 64, 8, 4)                                     \
        ENGRAM_NORM_CASE(FN, 64, 16, 3) ENGRAM_NORM_CASE(FN, 64, 16, 4)                                   \
    }

}  // namespace
}  // namespace engram
