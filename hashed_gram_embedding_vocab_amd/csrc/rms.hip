// rms.hip -- RMS norm of the residual stream's rows with the residual's addition,
// in the plan's type and / or in 8 bits with a scale for each 128 channels, and
// its gradients.
//
//   s = x + r (rounded to the plan's type),  rr = (mean(s^2) + eps)^(-1/2),  y = s rr gamma
//   in 8 bits: sc = the smallest power of two >= 2^-126 with amax(|y|) / sc <= 448, q = y / sc in e4m3
//   with g = dy gamma and s' = s rr:
//   dx = rr (g - s' mean(g s')) + ds,  dgamma = sum dy s'
//
// y is kept in fp32 until it is rounded once, to the plan's type and to e4m3
// each on its own.  s is rounded first because it is what the residual stream
// holds: the norm and its gradient then see the values that the next layer and
// the backward read.
//
// Rows are spread and walked as in norm.hip, the next row's loads in flight while a row
// is worked on: both kernels are bound by memory.  d = 2560 in bf16 with a residual:
// 32,768 rows in both types 141 us, 5.3 TB/s (a copy of 2 GB runs at 4.9 TB/s here), in
// fp32 to fp32 263 us, 5.1 TB/s; gradients of 131,072 rows 512 us, 5.2 TB/s.  256 rows in 8 bits 5.2 us: a launch
// and one trip to memory and back.
#include <algorithm>

#include "block8.h"
#include "engram_internal.h"
#include "rows.h"
#include "vec8.h"

namespace engram {
namespace {

// a + b in fp32 rounded to T, as loaded from memory
__device__ __forceinline__ Raw8<uint16_t> add8(const Raw8<uint16_t> &a, const Raw8<uint16_t> &b) {
    const F8 x = a.get(), y = b.get();
    Raw8<uint16_t> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16x2(x.v[2 * i] + y.v[2 * i], x.v[2 * i + 1] + y.v[2 * i + 1]);
    return r;
}
__device__ __forceinline__ Raw8<float> add8(const Raw8<float> &a, const Raw8<float> &b) {
    return Raw8<float>{a.a + b.a, a.b + b.b};
}
__device__ __forceinline__ void store_raw8(uint16_t *p, const Raw8<uint16_t> &x) {
    *reinterpret_cast<u32x4_t *>(p) = x.w;
}
__device__ __forceinline__ void store_raw8(float *p, const Raw8<float> &x) {
    *reinterpret_cast<f32x4_t *>(p) = x.a;
    *reinterpret_cast<f32x4_t *>(p + 4) = x.b;
}

// Largest finite magnitude of a block, over the lanes that hold it (16; 8 where
// a row has 64 channels at most).
template <int L>
__device__ __forceinline__ uint32_t block_top(const F8 &y) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_bits(y.v[i]));
    m = dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(m)));
    if constexpr (L >= 16) m = dpp_max<0x140>(m);
    return m;
}

// KEEP: gamma stays in registers (not where 16 waves of 128 registers share a row).
template <typename T, int L, int W, int NCH, bool RES>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rms_kernel(const T *x, const T *res, int64_t n_rows, int32_t d,
                                                                   const float *gamma, float eps, T *total, T *y,
                                                                   uint8_t *q, uint8_t *scales, float *rrms) {
    constexpr bool KEEP = W < 16;
    __shared__ float red[2][1][W];
    const Rows<L, W> at;
    const int64_t stride = (int64_t)gridDim.x * at.kAtOnce;
    const int32_t kb_all = (d + 127) / 128, pitch = (kb_all + 3) / 4 * 4;
    int turn = 0;
    const float inv_d = 1.f / (float)d;
    F8 g[KEEP ? NCH : 1];
    Raw8<T> next[NCH], next_r[RES ? NCH : 1];
    int64_t r = (int64_t)blockIdx.x * at.kAtOnce + at.slot;
    const int64_t r_wave = r - (L < 64 ? at.lane / L : 0);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = at.c0 + 512 * W * j;
        const int64_t o = min(r, n_rows - 1) * d + c;
        next[j] = Raw8<T>{};
        if constexpr (RES) next_r[j] = Raw8<T>{};
        if (c < d) {
            next[j] = load_raw8(x + o);
            if constexpr (RES) next_r[j] = load_raw8(res + o);
        }
        if constexpr (KEEP) {
            g[j] = F8{};
            if (c < d) g[j] = load8(gamma + c);
        }
    }
    for (int64_t k = r_wave; k < n_rows; k += stride, r += stride) {
        F8 v[NCH];
        const int64_t rn = min(r + stride, n_rows - 1);
        const bool live = L == 64 || r < n_rows;
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            Raw8<T> raw = next[j];
            if constexpr (RES) raw = add8(raw, next_r[j]);
            if (c < d) {
                next[j] = load_raw8(x + rn * d + c);
                if constexpr (RES) {
                    next_r[j] = load_raw8(res + rn * d + c);
                    if (live) store_raw8(total + r * d + c, raw);
                }
            }
            v[j] = raw.get();
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] += v[j].v[i] * v[j].v[i];
        }
        row_sums<L, W>(s, &red, at.wave, at.lane, turn);
        const float rr = 1.f / sqrtf(s[0] * inv_d + eps);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            F8 gj = {};
            if constexpr (KEEP)
                gj = g[j];
            else if (c < d)
                gj = load8(gamma + c);
            F8 o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o.v[i] = c < d ? v[j].v[i] * rr * gj.v[i] : 0.f;
            if (y && c < d && live) store8(y + r * d + c, o);
            if (q) {  // (the same for all lanes: a block's lanes take part together)
                const uint32_t byte = scale_byte(block_top<L>(o));
                if (c < d && live) *reinterpret_cast<u32x2_t *>(q + r * d + c) = cvt8(o, scale_inverse(byte));
                // a block's first lane stores its scale; rows end with ones
                const int32_t kb = c >> 7;
                if ((c & 127) == 0 && live) {
                    if (kb < pitch) scales[r * pitch + kb] = kb < kb_all ? (uint8_t)byte : (uint8_t)127;
                    if constexpr (L < 64) {  // up to two blocks: their lanes do not reach the row's end
                        if (kb == 0)
                            for (int32_t z = L / 16 > 1 ? L / 16 : 1; z < pitch; ++z) scales[r * pitch + z] = 127;
                    }
                }
            }
        }
        if (at.lane % L == 0 && at.wave == 0 && live && rrms) rrms[r] = rr;
    }
}

// A block's rows' dgamma sums end as one row of `part` [blocks][d], or, where the
// launch is one block, in dgamma itself.
template <typename T, int L, int W, int NCH, bool RES>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rms_bwd_kernel(const T *x, const T *dy, const T *ds,
                                                                       int64_t n_rows, int32_t d, const float *gamma,
                                                                       const float *rrms, T *dx, float *part,
                                                                       bool accumulate, float *dgamma) {
    __shared__ float red[2][1][W];
    __shared__ float sum_s[W == 1 ? 4 : 1][W == 1 ? NCH * 512 : 1];
    const Rows<L, W> at;
    const int64_t stride = (int64_t)gridDim.x * at.kAtOnce;
    int turn = 0;
    const float inv_d = 1.f / (float)d;
    F8 gm[NCH], dg[NCH];
    Raw8<T> xn[NCH], yn[NCH], sn[RES ? NCH : 1];
    int64_t r = (int64_t)blockIdx.x * at.kAtOnce + at.slot;
    const int64_t r_wave = r - (L < 64 ? at.lane / L : 0);
    float rr_n = rrms[min(r, n_rows - 1)];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = at.c0 + 512 * W * j;
        const int64_t o = min(r, n_rows - 1) * d + c;
        gm[j] = dg[j] = F8{};
        xn[j] = yn[j] = Raw8<T>{};
        if constexpr (RES) sn[j] = Raw8<T>{};
        if (c < d) {
            xn[j] = load_raw8(x + o);
            yn[j] = load_raw8(dy + o);
            if constexpr (RES) sn[j] = load_raw8(ds + o);
            gm[j] = load8(gamma + c);
        }
    }
    for (int64_t k = r_wave; k < n_rows; k += stride, r += stride) {
        Raw8<T> xr[NCH], yr[NCH], sr[RES ? NCH : 1];
        const float rr = rr_n;
        const int64_t rn = min(r + stride, n_rows - 1);
        rr_n = rrms[rn];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            xr[j] = xn[j];
            yr[j] = yn[j];
            if constexpr (RES) sr[j] = sn[j];
            if (c < d) {
                xn[j] = load_raw8(x + rn * d + c);
                yn[j] = load_raw8(dy + rn * d + c);
                if constexpr (RES) sn[j] = load_raw8(ds + rn * d + c);
            }
        }
        const bool live = L == 64 || r < n_rows;
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (at.c0 + 512 * W * j < d && live) {
                const F8 xv = xr[j].get(), yv = yr[j].get();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float t = yv.v[i] * (xv.v[i] * rr);
                    dg[j].v[i] += t;
                    s[0] += t * gm[j].v[i];
                }
            }
        }
        row_sums<L, W>(s, &red, at.wave, at.lane, turn);
        const float m = s[0] * inv_d;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            if (c < d) {
                const F8 xv = xr[j].get(), yv = yr[j].get();
                F8 o;
#pragma unroll
                for (int i = 0; i < 8; ++i) o.v[i] = rr * (yv.v[i] * gm[j].v[i] - xv.v[i] * rr * m);
                if constexpr (RES) {
                    const F8 sv = sr[j].get();
#pragma unroll
                    for (int i = 0; i < 8; ++i) o.v[i] += sv.v[i];
                }
                store8(dx + r * d + c, o);
            }
        }
    }
    if constexpr (W == 1) {
        // the sums of the block's rows at once, in slot order
        const int w = threadIdx.x >> 6;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum_s[w][(j * 8 + i) * 64 + at.lane] = dg[j].v[i];
        __syncthreads();
        // value (j, i, lane) of a wave's image is channel (j * 64 + lane % L) * 8 + i
        for (int k = threadIdx.x; k < d; k += 256) {
            const int at0 = ((k >> 9) * 8 + (k & 7)) * 64 + (k >> 3) % 64;
            float t = 0.f;
#pragma unroll
            for (int ww = 0; ww < 4; ++ww)
#pragma unroll
                for (int l = 0; l < 64; l += L) t += sum_s[ww][at0 + l];
            if (gridDim.x > 1)
                part[(int64_t)blockIdx.x * d + k] = t;
            else
                dgamma[k] = accumulate ? dgamma[k] + t : t;
        }
    } else {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = at.c0 + 512 * W * j;
            if (c < d) {
                if (gridDim.x > 1) {
                    store8(part + (int64_t)blockIdx.x * d + c, dg[j]);
                } else {
                    F8 s = dg[j];
                    if (accumulate) {
                        const F8 old = load8(dgamma + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) s.v[i] = old.v[i] + s.v[i];
                    }
                    store8(dgamma + c, s);
                }
            }
        }
    }
}

template <typename T, bool RES>
void rms_fwd(const RmsArgs &a, hipStream_t s) {
    const RowShape sh = row_shape(a.d);
    const int64_t blocks = norm_blocks(sh, a.n_rows, sh.steps == 1 ? 8 : sh.steps == 2 ? 4 : 2);
#define ENGRAM_RMS_FWD(L, W, N)                                                                                     \
    launch_kernel((rms_kernel<T, L, W, N, RES>), dim3((unsigned)blocks), dim3(W == 1 ? 256 : 64 * W), s,            \
                  static_cast<const T *>(a.x), static_cast<const T *>(a.res), a.n_rows, a.d, a.gamma, a.eps,        \
                  static_cast<T *>(a.total), static_cast<T *>(a.y), a.q, a.scales, a.rrms)
    ENGRAM_NORM_SWITCH(ENGRAM_RMS_FWD, sh)
#undef ENGRAM_RMS_FWD
}

template <typename T, bool RES>
void rms_bwd(const RmsArgs &a, hipStream_t s) {
    const RowShape sh = row_shape(a.d);
    const int32_t blocks = rms_bwd_blocks(a.n_rows, a.d);
#define ENGRAM_RMS_BWD(L, W, N)                                                                                     \
    launch_kernel((rms_bwd_kernel<T, L, W, N, RES>), dim3((unsigned)blocks), dim3(W == 1 ? 256 : 64 * W), s,        \
                  static_cast<const T *>(a.x), static_cast<const T *>(a.dy), static_cast<const T *>(a.ds),          \
                  a.n_rows, a.d, a.gamma, a.rrms, static_cast<T *>(a.dx), a.part, a.accumulate, a.dgamma)
    ENGRAM_NORM_SWITCH(ENGRAM_RMS_BWD, sh)
#undef ENGRAM_RMS_BWD
    if (blocks > 1)
        launch_kernel(norm_bwd_sum_kernel, dim3((unsigned)((a.d + 63) / 64), 1), dim3(1024), s, a.part, blocks, a.d,
                      a.accumulate, a.dgamma, static_cast<float *>(nullptr));
}

}  // namespace

int32_t rms_bwd_blocks(int64_t n_rows, int32_t d) {
    const RowShape sh = row_shape(d);
    // four rows a wave take less than the second launch
    if (n_rows <= 4 * sh.at_once()) return 1;
    return (int32_t)norm_blocks(sh, n_rows, sh.steps == 1 ? 4 : 2);
}

void launch_rms(engram_dtype dt, const RmsArgs &a, hipStream_t s) {
    if (dt == ENGRAM_BF16) {
        if (a.res)
            rms_fwd<uint16_t, true>(a, s);
        else
            rms_fwd<uint16_t, false>(a, s);
    } else {
        if (a.res)
            rms_fwd<float, true>(a, s);
        else
            rms_fwd<float, false>(a, s);
    }
}

void launch_rms_bwd(engram_dtype dt, const RmsArgs &a, hipStream_t s) {
    if (dt == ENGRAM_BF16) {
        if (a.ds)
            rms_bwd<uint16_t, true>(a, s);
        else
            rms_bwd<uint16_t, false>(a, s);
    } else {
        if (a.ds)
            rms_bwd<float, true>(a, s);
        else
            rms_bwd<float, false>(a, s);
    }
}

}  // namespace engram
