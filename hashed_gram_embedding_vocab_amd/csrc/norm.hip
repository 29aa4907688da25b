// norm.hip -- layer norm of the hidden state's rows and its gradients.
//
//   y = (x - mean) rstd gamma + beta,  rstd = (mean((x - mean)^2) + eps)^(-1/2)
//   with g = dy gamma and x' = (x - mean) rstd:
//   dx = rstd (g - mean(g) - x' mean(g x')),  dgamma = sum dy x',  dbeta = sum dy
//
// A row of d channels is held in the registers of W waves, 8 channels a lane
// and step, NCH steps: x is read once, the variance is the mean square of
// the centred values (not a difference of two sums), all in fp32.
#include <algorithm>

#include "engram_internal.h"
#include "vec8.h"

namespace engram {
namespace {

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
    return x;
}

// Sums over the W waves of a row.  `turn` alternates between two LDS slots,
// so one barrier a sum is enough: a slot is written again only after the
// barrier of the sum in between.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*red)[2][N][W], int wave, int lane, int &turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
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

// blockDim = 256 (four rows) where W == 1, else 64 W (one row).
template <typename T, int W, int NCH>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_kernel(const T *x, int64_t n_rows, int32_t d,
                                                                     const float *gamma, const float *beta, float eps,
                                                                     T *y, float *mean, float *rstd) {
    __shared__ float red[2][1][W];
    const int lane = threadIdx.x & 63, wave = W == 1 ? 0 : threadIdx.x >> 6;
    const int rows_per_block = W == 1 ? 4 : 1;
    int turn = 0;
    const float inv_d = 1.f / (float)d;
    for (int64_t r = (int64_t)blockIdx.x * rows_per_block + (W == 1 ? threadIdx.x >> 6 : 0); r < n_rows;
         r += (int64_t)gridDim.x * rows_per_block) {
        F8 v[NCH];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = ((j * W + wave) * 64 + lane) * 8;
            v[j] = F8{};
            if (c < d) v[j] = load8(x + r * d + c);
        }
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] += v[j].v[i];
        row_sums<W>(s, &red, wave, lane, turn);
        const float mu = s[0] * inv_d;
        s[0] = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = ((j * W + wave) * 64 + lane) * 8;
            if (c < d)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[j].v[i] -= mu;
                    s[0] += v[j].v[i] * v[j].v[i];
                }
        }
        row_sums<W>(s, &red, wave, lane, turn);
        const float rs = 1.f / sqrtf(s[0] * inv_d + eps);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = ((j * W + wave) * 64 + lane) * 8;
            if (c < d) {
                const F8 g = load8(gamma + c);
                F8 o;
#pragma unroll
                for (int i = 0; i < 8; ++i) o.v[i] = v[j].v[i] * rs * g.v[i];
                if (beta) {
                    const F8 b = load8(beta + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o.v[i] += b.v[i];
                }
                store8(y + r * d + c, o);
            }
        }
        if (lane == 0 && wave == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

// Each block walks the rows blockIdx, blockIdx + gridDim, ... (of its four
// waves where W == 1) and keeps its channels' dgamma and dbeta sums in
// registers; they end as one row of `part` [2][blocks][d].
template <typename T, int W, int NCH>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_bwd_kernel(const T *x, const T *dy, int64_t n_rows,
                                                                         int32_t d, const float *gamma,
                                                                         const float *mean, const float *rstd, T *dx,
                                                                         float *part) {
    __shared__ float red[2][2][W];
    __shared__ float sum_s[W == 1 ? 4 : 1][W == 1 ? NCH * 512 : 1];
    const int lane = threadIdx.x & 63, wave = W == 1 ? 0 : threadIdx.x >> 6;
    const int slot = W == 1 ? threadIdx.x >> 6 : 0;
    constexpr int kRows = W == 1 ? 4 : 1;
    int turn = 0;
    const float inv_d = 1.f / (float)d;
    F8 gm[NCH], dg[NCH], db[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = ((j * W + wave) * 64 + lane) * 8;
        gm[j] = dg[j] = db[j] = F8{};
        if (c < d) gm[j] = load8(gamma + c);
    }
    for (int64_t r = (int64_t)blockIdx.x * kRows + slot; r < n_rows; r += (int64_t)gridDim.x * kRows) {
        F8 xv[NCH], gv[NCH];
        const float mu = mean[r], rs = rstd[r];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = ((j * W + wave) * 64 + lane) * 8;
            xv[j] = gv[j] = F8{};
            if (c < d) {
                xv[j] = load8(x + r * d + c);
                gv[j] = load8(dy + r * d + c);
            }
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = ((j * W + wave) * 64 + lane) * 8;
            if (c < d)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (xv[j].v[i] - mu) * rs;
                    dg[j].v[i] += gv[j].v[i] * xh;
                    db[j].v[i] += gv[j].v[i];
                    const float g = gv[j].v[i] * gm[j].v[i];
                    s[0] += g;
                    s[1] += g * xh;
                    xv[j].v[i] = xh;
                    gv[j].v[i] = g;
                }
        }
        row_sums<W>(s, &red, wave, lane, turn);
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = ((j * W + wave) * 64 + lane) * 8;
            if (c < d) {
                F8 o;
#pragma unroll
                for (int i = 0; i < 8; ++i) o.v[i] = rs * (gv[j].v[i] - m1 - xv[j].v[i] * m2);
                store8(dx + r * d + c, o);
            }
        }
    }
    if constexpr (W == 1) {
        // the four waves' sums, in wave order
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NCH; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum_s[slot][(j * 8 + i) * 64 + lane] = q == 0 ? dg[j].v[i] : db[j].v[i];
            __syncthreads();
            // position (j, i, lane) of the image is channel (j * 64 + lane) * 8 + i
            for (int k = threadIdx.x; k < NCH * 512; k += 256) {
                const int j = k >> 9, l = (k >> 3) & 63, i = k & 7;
                const int at = (j * 8 + i) * 64 + l;
                if (k < d)
                    part[((int64_t)q * gridDim.x + blockIdx.x) * d + k] =
                        ((sum_s[0][at] + sum_s[1][at]) + sum_s[2][at]) + sum_s[3][at];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = ((j * W + wave) * 64 + lane) * 8;
            if (c < d) {
                store8(part + (int64_t)blockIdx.x * d + c, dg[j]);
                store8(part + ((int64_t)gridDim.x + blockIdx.x) * d + c, db[j]);
            }
        }
    }
}

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

// Waves per row: one while the backward's NCH stays at most 5 (about 200
// registers), more for wider rows.
struct RowShape {
    int waves, steps;
};
RowShape row_shape(int32_t d) {
    const int units = (d + 511) / 512;
    int w = 1;
    while (w < 16 && (units + w - 1) / w > (w == 1 ? 5 : 4)) w *= 2;
    return RowShape{w, (units + w - 1) / w};
}

#define ENGRAM_NORM_CASE(FN, W, N) \
    case W * 16 + N: FN(W, N); break;
#define ENGRAM_NORM_SWITCH(FN, SHAPE)                                               \
    switch ((SHAPE).waves * 16 + (SHAPE).steps) {                                   \
        ENGRAM_NORM_CASE(FN, 1, 1) ENGRAM_NORM_CASE(FN, 1, 2) ENGRAM_NORM_CASE(FN, 1, 3)   \
        ENGRAM_NORM_CASE(FN, 1, 4) ENGRAM_NORM_CASE(FN, 1, 5)                       \
        ENGRAM_NORM_CASE(FN, 2, 3) ENGRAM_NORM_CASE(FN, 2, 4)                       \
        ENGRAM_NORM_CASE(FN, 4, 3) ENGRAM_NORM_CASE(FN, 4, 4)                       \
        ENGRAM_NORM_CASE(FN, 8, 3) ENGRAM_NORM_CASE(FN, 8, 4)                       \
        ENGRAM_NORM_CASE(FN, 16, 3) ENGRAM_NORM_CASE(FN, 16, 4)                     \
    }

template <typename T>
void norm_fwd(const NormArgs &a, hipStream_t s) {
    const RowShape sh = row_shape(a.d);
    const int rows_per_block = sh.waves == 1 ? 4 : 1;
    const int64_t blocks = std::min<int64_t>((a.n_rows + rows_per_block - 1) / rows_per_block, (int64_t)1 << 20);
#define ENGRAM_NORM_FWD(W, N)                                                                                      \
    launch_kernel((norm_kernel<T, W, N>), dim3((unsigned)blocks), dim3(W == 1 ? 256 : 64 * W), s,                  \
                  static_cast<const T *>(a.x), a.n_rows, a.d, a.gamma, a.beta, a.eps, static_cast<T *>(a.y), a.mean, \
                  a.rstd)
    ENGRAM_NORM_SWITCH(ENGRAM_NORM_FWD, sh)
#undef ENGRAM_NORM_FWD
}

template <typename T>
void norm_bwd(const NormArgs &a, hipStream_t s) {
    const RowShape sh = row_shape(a.d);
    const int32_t blocks = norm_bwd_blocks(a.n_rows, a.d);
#define ENGRAM_NORM_BWD(W, N)                                                                                     \
    launch_kernel((norm_bwd_kernel<T, W, N>), dim3((unsigned)blocks), dim3(W == 1 ? 256 : 64 * W), s,             \
                  static_cast<const T *>(a.x), static_cast<const T *>(a.dy), a.n_rows, a.d, a.gamma, a.mean,      \
                  a.rstd, static_cast<T *>(a.dx), a.part)
    ENGRAM_NORM_SWITCH(ENGRAM_NORM_BWD, sh)
#undef ENGRAM_NORM_BWD
    launch_kernel(norm_bwd_sum_kernel, dim3((unsigned)((a.d + 63) / 64), 2), dim3(1024), s, a.part, blocks, a.d,
                  a.accumulate, a.dgamma, a.dbeta);
}

}  // namespace

bool norm_fits(int32_t d) { return d <= 16 * 4 * 512; }

int32_t norm_bwd_blocks(int64_t n_rows, int32_t d) {
    const RowShape sh = row_shape(d);
    const int rows_per_block = sh.waves == 1 ? 4 : 1;
    const int64_t most = sh.waves <= 2 ? 512 : sh.waves == 4 ? 512 : 256;
    return (int32_t)std::min<int64_t>((n_rows + rows_per_block - 1) / rows_per_block, most);
}

void launch_norm(engram_dtype dt, const NormArgs &a, hipStream_t s) {
    if (dt == ENGRAM_BF16)
        norm_fwd<uint16_t>(a, s);
    else
        norm_fwd<float>(a, s);
}

void launch_norm_bwd(engram_dtype dt, const NormArgs &a, hipStream_t s) {
    if (dt == ENGRAM_BF16)
        norm_bwd<uint16_t>(a, s);
    else
        norm_bwd<float>(a, s);
}

}  // namespace engram
