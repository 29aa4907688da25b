// fp8.hip -- the matrix product in 8-bit floating point (e4m3) with a scale
// for each block of 128, and the quantisation that makes its operands.
//
//   s = the smallest power of two >= 2^-126 with amax(block) / s <= 448
//   q = x / s rounded to nearest-even e4m3
//   C[m][n] = sum over blocks kb of  sa[m][kb] sb[n][kb]  sum_{k in kb} a[m][k] b[n][k]
//
// Scales are stored as their biased exponents (e8m0 bytes), which is the
// form the gfx950 scaled matrix instruction multiplies by itself:
// v_mfma_scale_f32_16x16x128_f8f6f4 covers exactly one block of 128 along K,
// so the scales cost no vector arithmetic and the accumulators stay fp32
// across blocks.  A power of two also makes x / s exact: the quantised values
// do not depend on how a division rounds.
//
// The 8-bit matrix instructions add the products of one block with about 13
// bits below the largest of them (measured: beside a product of 1, one of
// 2^-13 counts and one of 2^-14 is lost), which puts the result 1.5e-5 of its
// norm off: far below bf16's rounding (2^-9 on average 1.7e-3 of the norm),
// but not what fp32 is asked for.  So a bf16 result takes them, and an fp32
// result expands e4m3 times its scale to bf16 in registers (both exact) and
// takes the bf16 matrix instructions, whose sums are fp32 throughout (1e-8
// measured), at half the matrix rate.
#include <algorithm>

#include "engram_internal.h"
#include "vec8.h"

namespace engram {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- quantisation
// |x| as bits, 0 where x is not finite
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// Biased exponent of the block's scale from the bits of its largest finite
// magnitude (448 = 1.75 * 2^8).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(e, 1);
}

// 1 / scale: exact (a power of two in the normal range, 2^-120 .. 2^126)
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two values to e4m3 bytes.  Finite values are at most 448 here; infinities
// have no e4m3 form and become NaN like NaNs.
__device__ __forceinline__ float no_inf(float x) {
    return (__float_as_uint(x) & 0x7FFFFFFFu) == 0x7F800000u ? __uint_as_float(0x7FC00000u) : x;
}
template <bool HI>
__device__ __forceinline__ uint32_t cvt2(float a, float b, uint32_t old) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(no_inf(a), no_inf(b), (int)old, HI);
}
__device__ __forceinline__ u32x2_t cvt8(const F8 &x, float inv) {
    u32x2_t q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w = cvt2<false>(x.v[4 * i] * inv, x.v[4 * i + 1] * inv, 0u);
        q[i] = cvt2<true>(x.v[4 * i + 2] * inv, x.v[4 * i + 3] * inv, w);
    }
    return q;
}

// 8 values at column c of a row of `cols`, zeros past its end.  VEC: rows are
// whole 8-value units and 16-byte aligned.
template <bool VEC, typename T>
__device__ __forceinline__ F8 load_cols(const T *row, int64_t c, int64_t cols) {
    F8 x = {};
    if constexpr (VEC) {
        if (c < cols) x = load8(row + c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) {
                if constexpr (sizeof(T) == 2)
                    x.v[i] = bf16_to_f32(row[c + i]);
                else
                    x.v[i] = row[c + i];
            }
    }
    return x;
}

template <bool VEC>
__device__ __forceinline__ void store_cols(uint8_t *row, int64_t c, int64_t cols, u32x2_t q) {
    if constexpr (VEC) {
        if (c < cols) *reinterpret_cast<u32x2_t *>(row + c) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
    }
}

// One wave per (row, 512 columns): a block is 16 lanes, and the wave's four
// scale bytes are one word of the scales' row (its blocks past the last hold 127, i.e. one).
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T *x, int64_t rows, int64_t cols, uint8_t *q,
                                                            uint8_t *scales) {
    const int lane = threadIdx.x & 63;
    const int64_t strips = (cols + 511) / 512, n_items = rows * strips;
    const int64_t kb = (cols + 127) / 128;
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < n_items; item += (int64_t)gridDim.x * 4) {
        const int64_t r = item / strips, strip = item - r * strips;
        const int64_t c = strip * 512 + lane * 8;
        const F8 v = load_cols<VEC>(x + r * cols, c, cols);
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, finite_bits(v.v[i]));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
        const uint32_t byte = scale_byte(top);
        store_cols<VEC>(q + r * cols, c, cols, cvt8(v, scale_inverse(byte)));
        const uint32_t mine = strip * 4 + (lane >> 4) < kb ? byte : 127u;
        uint32_t word = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) word |= (uint32_t)__builtin_amdgcn_readlane((int)mine, 16 * i) << (8 * i);
        if (lane == 0) *reinterpret_cast<uint32_t *>(scales + (r * strips + strip) * 4) = word;
    }
}

// One workgroup per 128 x 128 tile of x, 64 values a thread (8 rows x 8
// columns).  TR: q is [cols][rows], its blocks run along x's rows.
// BLOCK_ROWS 128: one scale for the tile; 1 (TR only): one per column of x.
template <typename T, bool VEC, bool TR, int BLOCK_ROWS>
__global__ __launch_bounds__(256) void quantize_tile_kernel(const T *x, int64_t rows, int64_t cols, uint8_t *q,
                                                            uint8_t *scales) {
    static_assert(TR || BLOCK_ROWS == 128, "rows of their own scale go through quantize_rows_kernel");
    constexpr int kPitch = 128 + 16;
    __shared__ uint32_t top_s[4][BLOCK_ROWS == 1 ? 128 : 1];
    __shared__ __attribute__((aligned(16))) uint8_t tile[TR ? 128 * kPitch : 16];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // 8 columns from 8 cg, 8 rows from 8 rg
    const int64_t col_tiles = (cols + 127) / 128, row_tiles = (rows + 127) / 128;
    for (int64_t tl = blockIdx.x; tl < col_tiles * row_tiles; tl += gridDim.x) {
        const int64_t tr = tl / col_tiles, tc = tl - tr * col_tiles;
        const int64_t r0 = tr * 128, c0 = tc * 128;
        F8 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t r = r0 + 8 * rg + j;
            v[j] = F8{};
            if (r < rows) v[j] = load_cols<VEC>(x + r * cols, c0 + 8 * cg, cols);
        }
        uint32_t top[8];  // of this thread's columns
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top[i] = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) top[i] = max(top[i], finite_bits(v[j].v[i]));
        }
        if constexpr (BLOCK_ROWS == 128) {
#pragma unroll
            for (int i = 1; i < 8; ++i) top[0] = max(top[0], top[i]);
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) top[0] = max(top[0], (uint32_t)__shfl_xor((int)top[0], off));
            if (lane == 0) top_s[w][0] = top[0];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                top[i] = max(top[i], (uint32_t)__shfl_xor((int)top[i], 16));
                top[i] = max(top[i], (uint32_t)__shfl_xor((int)top[i], 32));
                if (lane < 16) top_s[w][8 * cg + i] = top[i];
            }
        }
        __syncthreads();
        uint32_t byte[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = BLOCK_ROWS == 1 ? 8 * cg + i : 0;
            byte[i] = scale_byte(max(max(top_s[0][at], top_s[1][at]), max(top_s[2][at], top_s[3][at])));
        }
        // the scales' rows are filled up with ones to whole words
        const int64_t kb_all = TR ? row_tiles : col_tiles, pitch = (kb_all + 3) / 4 * 4;
        const int64_t kb = TR ? tr : tc;
        const int pad = kb == kb_all - 1 ? (int)(pitch - kb_all) : 0;
        if constexpr (BLOCK_ROWS == 1) {
            if (rg == 0)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t row = c0 + 8 * cg + i;
                    if (row < cols) {
                        scales[row * pitch + kb] = (uint8_t)byte[i];
                        for (int z = 1; z <= pad; ++z) scales[row * pitch + kb + z] = 127;
                    }
                }
        } else if (threadIdx.x == 0) {
            const int64_t row = TR ? tc : tr;
            scales[row * pitch + kb] = (uint8_t)byte[0];
            for (int z = 1; z <= pad; ++z) scales[row * pitch + kb + z] = 127;
        }
        if constexpr (!TR) {
            const float inv = scale_inverse(byte[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t r = r0 + 8 * rg + j;
                if (r < rows) store_cols<VEC>(q + r * cols, c0 + 8 * cg, cols, cvt8(v[j], inv));
            }
            __syncthreads();  // top_s is rewritten by the next tile
        } else {
            // q^T through LDS: 8 bytes per column of x, then 16-byte pieces of q's rows
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                F8 col;
#pragma unroll
                for (int j = 0; j < 8; ++j) col.v[j] = v[j].v[i];
                *reinterpret_cast<u32x2_t *>(&tile[(8 * cg + i) * kPitch + 8 * rg]) =
                    cvt8(col, scale_inverse(byte[i]));
            }
            __syncthreads();
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int i = p * 256 + threadIdx.x;
                const int row = i >> 3, piece = (i & 7) * 16;
                const int64_t qr = c0 + row, qc = r0 + piece;
                if (qr >= cols || qc >= rows) continue;
                const u32x4_t b = *reinterpret_cast<const u32x4_t *>(&tile[row * kPitch + piece]);
                uint8_t *dst = q + qr * rows + qc;
                if (rows % 16 == 0) {
                    *reinterpret_cast<u32x4_t *>(dst) = b;
                } else {
#pragma unroll
                    for (int z = 0; z < 16; ++z)
                        if (qc + z < rows) dst[z] = (uint8_t)(b[z >> 2] >> (8 * (z & 3)));
                }
            }
            __syncthreads();  // tile and top_s are rewritten by the next tile
        }
    }
}

template <typename T, bool VEC>
void quantize(const QuantArgs &a, hipStream_t s) {
    const T *x = static_cast<const T *>(a.x);
    uint8_t *q = static_cast<uint8_t *>(a.q);
    const int64_t most = (int64_t)1 << 22;  // a launch holds fewer than 2^32 threads
    if (a.block_rows == 1 && !a.transpose) {
        const int64_t items = a.rows * ((a.cols + 511) / 512);
        launch_kernel((quantize_rows_kernel<T, VEC>), dim3((unsigned)std::min((items + 3) / 4, most)), dim3(256), s, x,
                      a.rows, a.cols, q, a.scales);
        return;
    }
    const dim3 grid((unsigned)std::min((a.rows + 127) / 128 * ((a.cols + 127) / 128), most));
    if (!a.transpose)
        launch_kernel((quantize_tile_kernel<T, VEC, false, 128>), grid, dim3(256), s, x, a.rows, a.cols, q, a.scales);
    else if (a.block_rows == 128)
        launch_kernel((quantize_tile_kernel<T, VEC, true, 128>), grid, dim3(256), s, x, a.rows, a.cols, q, a.scales);
    else
        launch_kernel((quantize_tile_kernel<T, VEC, true, 1>), grid, dim3(256), s, x, a.rows, a.cols, q, a.scales);
}

// ---------------------------------------------------------------- product
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// The MFMA's A side is rows of b (n), its B side rows of a (m), both
// K-contiguous: lane l holds row l % 16 and 32 of the block's 128 bytes, and
// result lane l holds C[m = l % 16][n = 4 (l / 16) .. + 3].  Which 32 bytes a
// lane group takes does not matter as long as both sides agree (the sum runs
// over the whole block): pieces (l / 16) and (l / 16) + 4 of 16 bytes.
struct Frag {
    u32x4_t half[2];
};

__device__ __forceinline__ Frag load_frag(const uint8_t *row, int64_t k, int64_t K, int lane) {
    Frag f = {};
    const int64_t p = k + 16 * (lane >> 4);
    if (p < K) f.half[0] = *reinterpret_cast<const u32x4_t *>(row + p);
    if (p + 64 < K) f.half[1] = *reinterpret_cast<const u32x4_t *>(row + p + 64);
    return f;
}

__device__ __forceinline__ i32x8_t e4m3x32(const Frag &f) {
    const u32x4_t &a = f.half[0], &b = f.half[1];
    return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Eight e4m3 values (two words) times 2^(byte - 127), as bf16.
__device__ __forceinline__ bf16x8_t to_bf16x8(uint32_t w0, uint32_t w1, uint32_t byte) {
    const float s = __uint_as_float(byte << 23);
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 128 x 128 outputs per workgroup, 64 x 64 per wave, operands from global memory.
template <bool F32>
__global__ __launch_bounds__(256) void product_kernel(ProductArgs g) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * 128 + 64 * (w & 1), m0 = (int64_t)blockIdx.y * 128 + 64 * (w >> 1);
    const int64_t kb = (g.K + 127) / 128, pitch = (kb + 3) / 4 * 4;
    const uint8_t *ar[4], *br[4], *as[4], *bs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = min(m0 + 16 * i + (lane & 15), g.M - 1), n = min(n0 + 16 * i + (lane & 15), g.N - 1);
        ar[i] = g.a + m * g.K;
        br[i] = g.b + n * g.K;
        as[i] = g.a_scales + m / g.a_block_rows * pitch;
        bs[i] = g.b_scales + n / g.b_block_rows * pitch;
    }
    f32x4_t acc[4][4] = {};
    for (int64_t k = 0; k < kb; ++k) {
        Frag fa[4], fb[4];
        uint32_t sa[4], sb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fa[i] = load_frag(ar[i], 128 * k, g.K, lane);
            fb[i] = load_frag(br[i], 128 * k, g.K, lane);
            sa[i] = as[i][k];
            sb[i] = bs[i][k];
        }
        if constexpr (F32) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8_t ha[4], hb[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int h = q >> 1, o = 2 * (q & 1);
                    ha[i] = to_bf16x8(fa[i].half[h][o], fa[i].half[h][o + 1], sa[i]);
                    hb[i] = to_bf16x8(fb[i].half[h][o], fb[i].half[h][o + 1], sb[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hb[i], ha[j], acc[i][j], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        e4m3x32(fb[i]), e4m3x32(fa[j]), acc[i][j], 0, 0, 0, (int)sb[i], 0, (int)sa[j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + 16 * i + 4 * (lane >> 4) + r;
                if (m >= g.M || n >= g.N) continue;
                if constexpr (F32)
                    static_cast<float *>(g.c)[m * g.N + n] = acc[i][j][r];
                else
                    static_cast<__bf16 *>(g.c)[m * g.N + n] = (__bf16)acc[i][j][r];
            }
        }
}

}  // namespace

void launch_quantize(engram_dtype dt, const QuantArgs &a, hipStream_t s) {
    // (q's rows are then whole 8-byte pieces too)
    const bool vec = a.cols % 8 == 0;
    if (dt == ENGRAM_BF16) {
        if (vec)
            quantize<uint16_t, true>(a, s);
        else
            quantize<uint16_t, false>(a, s);
    } else {
        if (vec)
            quantize<float, true>(a, s);
        else
            quantize<float, false>(a, s);
    }
}

size_t product_workspace(int64_t, int64_t, int64_t) { return 0; }

bool product_fits(int64_t M, int64_t N, int64_t) {
    return (M + 127) / 128 <= 65535 && (N + 127) / 128 < ((int64_t)1 << 24);
}

void launch_product(const ProductArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + 127) / 128), (unsigned)((a.M + 127) / 128));
    if (a.out_bf16)
        launch_kernel(product_kernel<false>, grid, dim3(256), s, a);
    else
        launch_kernel(product_kernel<true>, grid, dim3(256), s, a);
}

}  // namespace engram
