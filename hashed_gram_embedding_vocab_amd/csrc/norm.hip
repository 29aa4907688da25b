// norm.hip -- layer norm of the hidden state's rows and its gradients.
//
//   y = (x - mean) rstd gamma + beta,  rstd = (mean((x - mean)^2) + eps)^(-1/2)
//   with g = dy gamma and x' = (x - mean) rstd:
//   dx = rstd (g - mean(g) - x' mean(g x')),  dgamma = sum dy x',  dbeta = sum dy
//
// A row of d channels is held in the registers of W waves, 8 channels a lane
// and step, NCH steps (or of L lanes of one wave where d <= 8 L < 512): x is
// read once, the variance is the mean square of the centred values (not a
// difference of two sums), all in fp32.  Both kernels are bound by memory: a
// block walks many rows, so that gamma and beta (twice the bytes of a bf16 row)
// and the parameters' sums stay in registers, and the next row's loads are in
// flight while a row is worked on.  Measured in bf16 at d = 2560: forward of
// 32,768 rows 67 us (a block per four rows, gamma and beta read per row: 82),
// backward of 131,072 rows 388 us (one row at a time, expanded once: 467), 5.0
// and 5.2 TB/s; a large copy runs at 5.2.  Rows of 4096 to 16,384 channels (256 MB
// of them) run at 4.6 to 5.5 TB/s forward and 5.0 to 5.2 backward in bf16, 5.2 to
// 5.3 and 4.4 to 5.0 in fp32.
// Above 16,384 channels 16 waves share a row, which leaves a lane 128
// registers.  The forward then reads gamma and beta for every row (4.1 to 4.8
// TB/s).  The backward keeps its state all the same and spills 216 to 544 bytes
// a lane to scratch (in fp32 40 above 12,288 channels): 1.0 to 1.8 TB/s.
#include <algorithm>

#include "engram_internal.h"
#include "rows.h"
#include "vec8.h"

namespace engram {
namespace {

// KEEP: gamma and beta stay in registers (not where 16 waves of 128 registers
// share a row).
template <typename T, int L, int W, int NCH>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_kernel(const T *x, int64_t n_rows, int32_t d,
                                                                    const float *gamma, const float *beta, float eps,
                                                                    T *y, float *mean, float *rstd) {
    constexpr bool KEEP = W < 16;
    __shared__ float red[2][1][W];
    const Rows<L, W> at;
    const int64_t stride = (int64_t)gridDim.x * at.kAtOnce;
    int turn = 0;
    const float inv_d = 1.f / (float)d;
    F8 g[KEEP ? NCH : 1], b[KEEP ? NCH : 1];
    Raw8<T> next[NCH];
    // (where W == 1 a wave leaves when its rows end; rows of one wave may end
    // apart, and then stay on the last one without storing)
    int64_t r = (int64_t)blockIdx.x * at.kAtOnce + at.slot;
    const int64_t r_wave = r - (L < 64 ? at.lane / L : 0);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = at.c0 + 512 * W * j;
        next[j] = Raw8<T>{};
        if (c < d) next[j] = load_raw8(x + min(r, n_rows - 1) * d + c);
        if constexpr (KEEP) {
            g[j] = b[j] = F8{};
            if (c < d) {
                g[j] = load8(gamma + c);
                if (beta) b[j] = load8(beta + c);
            }
        }
    }
    for (int64_t k = r_wave; k < n_rows; k += stride, r += stride) {
        F8 v[NCH];
        const int64_t rn = min(r + stride, n_rows - 1);
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            v[j] = next[j].get();
            if (c < d) next[j] = load_raw8(x + rn * d + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] += v[j].v[i];
        }
        row_sums<L, W>(s, &red, at.wave, at.lane, turn);
        const float mu = s[0] * inv_d;
        s[0] = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (at.c0 + 512 * W * j < d)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[j].v[i] -= mu;
                    s[0] += v[j].v[i] * v[j].v[i];
                }
        }
        row_sums<L, W>(s, &red, at.wave, at.lane, turn);
        const float rs = 1.f / sqrtf(s[0] * inv_d + eps);
        if (L < 64 && r >= n_rows) continue;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            if (c < d) {
                F8 gj, bj = {};
                if constexpr (KEEP) {
                    gj = g[j];
                    bj = b[j];
                } else {
                    gj = load8(gamma + c);
                    if (beta) bj = load8(beta + c);
                }
                F8 o;
#pragma unroll
                for (int i = 0; i < 8; ++i) o.v[i] = v[j].v[i] * rs * gj.v[i] + bj.v[i];
                store8(y + r * d + c, o);
            }
        }
        if (at.lane % L == 0 && at.wave == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

// A block's rows' dgamma and dbeta sums end as one row of `part` [2][blocks][d],
// or, where the launch is one block, in dgamma and dbeta themselves.
// x and dy stay packed as loaded and are expanded twice (for the sums, for dx):
// expanded once they would take the registers of the next row's loads.
template <typename T, int L, int W, int NCH>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_bwd_kernel(const T *x, const T *dy, int64_t n_rows,
                                                                        int32_t d, const float *gamma,
                                                                        const float *mean, const float *rstd, T *dx,
                                                                        float *part, bool accumulate, float *dgamma,
                                                                        float *dbeta) {
    __shared__ float red[2][2][W];
    __shared__ float sum_s[W == 1 ? 4 : 1][W == 1 ? NCH * 512 : 1];
    const Rows<L, W> at;
    const int64_t stride = (int64_t)gridDim.x * at.kAtOnce;
    int turn = 0;
    const float inv_d = 1.f / (float)d;
    F8 gm[NCH], dg[NCH], db[NCH];
    Raw8<T> xn[NCH], yn[NCH];
    int64_t r = (int64_t)blockIdx.x * at.kAtOnce + at.slot;
    const int64_t r_wave = r - (L < 64 ? at.lane / L : 0);
    float mu_n = mean[min(r, n_rows - 1)], rs_n = rstd[min(r, n_rows - 1)];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = at.c0 + 512 * W * j;
        gm[j] = dg[j] = db[j] = F8{};
        xn[j] = yn[j] = Raw8<T>{};
        if (c < d) {
            xn[j] = load_raw8(x + min(r, n_rows - 1) * d + c);
            yn[j] = load_raw8(dy + min(r, n_rows - 1) * d + c);
            gm[j] = load8(gamma + c);
        }
    }
    for (int64_t k = r_wave; k < n_rows; k += stride, r += stride) {
        Raw8<T> xr[NCH], yr[NCH];
        const float mu = mu_n, rs = rs_n;
        const int64_t rn = min(r + stride, n_rows - 1);
        mu_n = mean[rn];
        rs_n = rstd[rn];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            xr[j] = xn[j];
            yr[j] = yn[j];
            if (c < d) {
                xn[j] = load_raw8(x + rn * d + c);
                yn[j] = load_raw8(dy + rn * d + c);
            }
        }
        const bool live = L == 64 || r < n_rows;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (at.c0 + 512 * W * j < d && live) {
                const F8 xv = xr[j].get(), yv = yr[j].get();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (xv.v[i] - mu) * rs, g = yv.v[i] * gm[j].v[i];
                    dg[j].v[i] += yv.v[i] * xh;
                    db[j].v[i] += yv.v[i];
                    s[0] += g;
                    s[1] += g * xh;
                }
            }
        }
        row_sums<L, W>(s, &red, at.wave, at.lane, turn);
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            if (c < d) {
                const F8 xv = xr[j].get(), yv = yr[j].get();
                F8 o;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (xv.v[i] - mu) * rs;
                    o.v[i] = rs * (yv.v[i] * gm[j].v[i] - m1 - xh * m2);
                }
                store8(dx + r * d + c, o);
            }
        }
    }
    if constexpr (W == 1) {
        // the sums of the block's rows at once, in slot order
        const int w = threadIdx.x >> 6;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NCH; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum_s[w][(j * 8 + i) * 64 + at.lane] = q == 0 ? dg[j].v[i] : db[j].v[i];
            __syncthreads();
            // value (j, i, lane) of a wave's image is channel (j * 64 + lane % L) * 8 + i
            for (int k = threadIdx.x; k < d; k += 256) {
                const int at0 = ((k >> 9) * 8 + (k & 7)) * 64 + (k >> 3) % 64;
                float t = 0.f;
#pragma unroll
                for (int ww = 0; ww < 4; ++ww)
#pragma unroll
                    for (int l = 0; l < 64; l += L) t += sum_s[ww][at0 + l];
                float *dst = q == 0 ? dgamma : dbeta;
                if (gridDim.x > 1)
                    part[((int64_t)q * gridDim.x + blockIdx.x) * d + k] = t;
                else if (dst)
                    dst[k] = accumulate ? dst[k] + t : t;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            if (c < d) {
                if (gridDim.x > 1) {
                    store8(part + (int64_t)blockIdx.x * d + c, dg[j]);
                    store8(part + ((int64_t)gridDim.x + blockIdx.x) * d + c, db[j]);
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float *dst = q == 0 ? dgamma : dbeta;
                        if (!dst) continue;
                        F8 s = q == 0 ? dg[j] : db[j];
                        if (accumulate) {
                            const F8 old = load8(dst + c);
#pragma unroll
                            for (int i = 0; i < 8; ++i) s.v[i] = old.v[i] + s.v[i];
                        }
                        store8(dst + c, s);
                    }
                }
            }
        }
    }
}

template <typename T>
void norm_fwd(const NormArgs &a, hipStream_t s) {
    const RowShape sh = row_shape(a.d);
    const int64_t blocks = norm_blocks(sh, a.n_rows, sh.steps == 1 ? 8 : sh.steps == 2 ? 4 : 2);
#define ENGRAM_NORM_FWD(L, W, N)                                                                                 \
    launch_kernel((norm_kernel<T, L, W, N>), dim3((unsigned)blocks), dim3(W == 1 ? 256 : 64 * W), s,             \
                  static_cast<const T *>(a.x), a.n_rows, a.d, a.gamma, a.beta, a.eps, static_cast<T *>(a.y),     \
                  a.mean, a.rstd)
    ENGRAM_NORM_SWITCH(ENGRAM_NORM_FWD, sh)
#undef ENGRAM_NORM_FWD
}

template <typename T>
void norm_bwd(const NormArgs &a, hipStream_t s) {
    const RowShape sh = row_shape(a.d);
    const int32_t blocks = norm_bwd_blocks(a.n_rows, a.d);
#define ENGRAM_NORM_BWD(L, W, N)                                                                                 \
    launch_kernel((norm_bwd_kernel<T, L, W, N>), dim3((unsigned)blocks), dim3(W == 1 ? 256 : 64 * W), s,         \
                  static_cast<const T *>(a.x), static_cast<const T *>(a.dy), a.n_rows, a.d, a.gamma, a.mean,     \
                  a.rstd, static_cast<T *>(a.dx), a.part, a.accumulate, a.dgamma, a.dbeta)
    ENGRAM_NORM_SWITCH(ENGRAM_NORM_BWD, sh)
#undef ENGRAM_NORM_BWD
    if (blocks > 1)
        launch_kernel(norm_bwd_sum_kernel, dim3((unsigned)((a.d + 63) / 64), 2), dim3(1024), s, a.part, blocks, a.d,
                  a.accumulate, a.dgamma, a.dbeta);
}

}  // namespace

bool norm_fits(int32_t d) { return d <= 16 * 4 * 512; }

int32_t norm_bwd_blocks(int64_t n_rows, int32_t d) {
    const RowShape sh = row_shape(d);
    // four rows a wave take less than the second launch
    if (n_rows <= 4 * sh.at_once()) return 1;
    return (int32_t)norm_blocks(sh, n_rows, sh.steps == 1 ? 4 : 2);
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
