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
// The 8-bit matrix instructions add eight consecutive products at a time, each
// cut to 13 bits below the largest of the eight (measured: beside a product of 1
// one of 2^-13 counts, one of 2^-14 is lost among the same eight and kept in any
// other), and those sums in fp32.  Eight products lose less than 7 * 2^-13 of
// their largest, so the result less than 8.5e-4 of the sum of the products'
// magnitudes, about a fifth of bf16's half step, and 1.5e-5 of its norm on random
// operands, beside 1.7e-3 for the rounding to bf16.  That is not what fp32 is
// asked for: so a bf16 result takes them, and an fp32 result expands e4m3 times
// its scale to bf16 in registers (both exact) and takes the bf16 matrix
// instructions, whose sums are fp32 throughout (1e-8 measured), at half the
// matrix rate.
#include <algorithm>
#include <type_traits>

#include "engram_internal.h"
#include "vec8.h"

namespace engram {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- quantisation
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

// Vectors at any address (the hardware splits an access where it has to):
// rows whose length is no multiple of the vector's.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ Raw8<uint16_t> load_any8(const uint16_t *p) {
    return Raw8<uint16_t>{*reinterpret_cast<const u32x4_any *>(p)};
}
__device__ __forceinline__ Raw8<float> load_any8(const float *p) {
    return Raw8<float>{*reinterpret_cast<const f32x4_any *>(p), *reinterpret_cast<const f32x4_any *>(p + 4)};
}

// 8 values at column c of a row of `cols`, zeros past its end.  VEC: rows are
// whole 8-value units and 16-byte aligned.
template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> load_cols(const T *row, int64_t c, int64_t cols) {
    Raw8<T> x = {};
    if constexpr (VEC) {
        if (c < cols) x = load_raw8(row + c);
    } else if (c + 8 <= cols) {
        x = load_any8(row + c);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (c + i < cols) {
                if constexpr (sizeof(T) == 2)
                    x.w[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
                else if (i < 4)
                    x.a[i & 3] = row[c + i];
                else
                    x.b[i & 3] = row[c + i];
            }
    }
    return x;
}

template <bool VEC>
__device__ __forceinline__ void store_cols(uint8_t *row, int64_t c, int64_t cols, u32x2_t q) {
    if constexpr (VEC) {
        if (c < cols) *reinterpret_cast<u32x2_t *>(row + c) = q;
    } else if (c + 8 <= cols) {
        *reinterpret_cast<u32x2_any *>(row + c) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}
// over the 16 lanes of a row (neighbours, quads, halves, the row's mirror)
__device__ __forceinline__ uint32_t max16(uint32_t x) { return dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(x)))); }

// One wave per (U rows, 512 columns): a block is 16 lanes, and the wave's four
// scale bytes of a row are one word of the scales' row (its blocks past the
// last hold 127, i.e. one).  Bound by memory; the U rows' loads are in flight
// together (32,768 x 1280 bf16: 22 us with four rows a wave, 30 with one).
template <typename T, bool VEC, int U>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T *x, int64_t rows, int64_t cols, uint8_t *q,
                                                            uint8_t *scales) {
    const int lane = threadIdx.x & 63;
    const int32_t strips = (int32_t)((cols + 511) / 512);
    const int64_t n_items = (rows + U - 1) / U * strips;
    const int64_t kb = (cols + 127) / 128;
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < n_items; item += (int64_t)gridDim.x * 4) {
        const int64_t group = quotient(item, strips), r0 = group * U, strip = item - group * strips;
        const int64_t c = strip * 512 + lane * 8;
        Raw8<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_cols<VEC>(x + min(r0 + u, rows - 1) * cols, c, cols);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u;
            if (r >= rows) break;
            const F8 f = v[u].get();
            Top8<T> t8;
            t8.add(v[u]);
            uint32_t top = max16(t8.all());
            if (__any(top >= kNotFinite)) {
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, finite_bits(f.v[i]));
                top = max16(m);
            }
            const uint32_t byte = scale_byte(top);
            store_cols<VEC>(q + r * cols, c, cols, cvt8(f, scale_inverse(byte)));
            const uint32_t mine = strip * 4 + (lane >> 4) < kb ? byte : 127u;
            uint32_t word = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) word |= (uint32_t)__builtin_amdgcn_readlane((int)mine, 16 * i) << (8 * i);
            if (lane == 0) *reinterpret_cast<uint32_t *>(scales + (r * strips + strip) * 4) = word;
        }
    }
}

// One workgroup per 128 x 128 tile of x, 64 values a thread (8 rows x 8
// columns), kept packed.  TR: q is [cols][rows], its blocks run along x's rows;
// the tiles are taken down x's rows in groups, so that what is written at a
// time are neighbouring pieces of q's rows (across x's columns the pieces lie
// a row of q apart).  Bound by memory: 32,768 x 2560 bf16 49 us transposed with a
// scale a column (80 with the tiles across and 8-way bank conflicts).  BLOCK_ROWS 128: one
// scale for the tile; 1 (TR only): one per column of x.
template <typename T, bool VEC, bool TR, int BLOCK_ROWS>
__global__ __launch_bounds__(256) void quantize_tile_kernel(const T *x, int64_t rows, int64_t cols, uint8_t *q,
                                                            uint8_t *scales) {
    static_assert(TR || BLOCK_ROWS == 128, "rows of their own scale go through quantize_rows_kernel");
    constexpr int kTops = BLOCK_ROWS == 1 ? 128 : 1;
    __shared__ __attribute__((aligned(16))) uint32_t top_s[2][kTops < 8 ? 8 : kTops];
    __shared__ __attribute__((aligned(16))) uint8_t tile[TR ? 128 * 128 : 16];
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // 8 columns from 8 cg, 8 rows from 8 rg
    const int64_t col_tiles = (cols + 127) / 128, row_tiles = (rows + 127) / 128;
    constexpr int64_t kGroup = 16;
    int turn = 0;
    for (int64_t tl = blockIdx.x; tl < col_tiles * row_tiles; tl += gridDim.x, turn ^= 1) {
        int64_t tr, tc;
        if constexpr (TR) {
            const int64_t grp = quotient(tl, (int32_t)(kGroup * col_tiles)), in = tl - grp * kGroup * col_tiles;
            const int64_t n = min(kGroup, row_tiles - grp * kGroup);
            tc = quotient(in, (int32_t)n);
            tr = grp * kGroup + in - tc * n;
        } else {
            tr = quotient(tl, (int32_t)col_tiles);
            tc = tl - tr * col_tiles;
        }
        const int64_t r0 = tr * 128, c0 = tc * 128;
        Raw8<T> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t r = r0 + 8 * rg + j;
            v[j] = Raw8<T>{};
            if (r < rows) v[j] = load_cols<VEC>(x + r * cols, c0 + 8 * cg, cols);
        }
        // (two sets in turn: this one was last read before the previous tile's barriers)
        if (threadIdx.x < kTops) top_s[turn][threadIdx.x] = 0u;
        Top8<T> top;
#pragma unroll
        for (int j = 0; j < 8; ++j) top.add(v[j]);
        __syncthreads();
        if (__any(top.all() >= kNotFinite)) {
            uint32_t m[8] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const F8 f = v[j].get();
#pragma unroll
                for (int i = 0; i < 8; ++i) m[i] = max(m[i], finite_bits(f.v[i]));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) atomicMax(&top_s[turn][BLOCK_ROWS == 1 ? 8 * cg + i : 0], m[i]);
        } else {
            if constexpr (BLOCK_ROWS == 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) atomicMax(&top_s[turn][8 * cg + i], top.column(i));
            } else {
                const uint32_t m = max16(top.all());
                if (cg == 0) atomicMax(&top_s[turn][0], m);
            }
        }
        __syncthreads();
        uint32_t byte[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) byte[i] = scale_byte(top_s[turn][BLOCK_ROWS == 1 ? 8 * cg + i : 0]);
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
                if (r < rows) store_cols<VEC>(q + r * cols, c0 + 8 * cg, cols, cvt8(v[j].get(), inv));
            }
        } else {
            // q^T through LDS: unit rg of 8 bytes of row 8 cg + i sits at place
            // rg ^ cg (16 lanes of a row group take 16 places), read back as
            // 16-byte pieces of q's rows
            F8 f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = v[j].get();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                F8 col;
#pragma unroll
                for (int j = 0; j < 8; ++j) col.v[j] = f[j].v[i];
                *reinterpret_cast<u32x2_t *>(&tile[(8 * cg + i) * 128 + (rg ^ cg) * 8]) =
                    cvt8(col, scale_inverse(byte[i]));
            }
            __syncthreads();
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int i = p * 256 + threadIdx.x;
                const int row = i >> 3, piece = i & 7, g = row >> 3;
                const int64_t qr = c0 + row, qc = r0 + piece * 16;
                if (qr >= cols || qc >= rows) continue;
                u32x4_t b = *reinterpret_cast<const u32x4_t *>(&tile[row * 128 + ((2 * piece) ^ (g & ~1)) * 8]);
                if (g & 1) b = u32x4_t{b[2], b[3], b[0], b[1]};
                uint8_t *dst = q + qr * rows + qc;
                if (rows % 16 == 0) {
                    *reinterpret_cast<u32x4_t *>(dst) = b;
                } else if (qc + 16 <= rows) {
                    *reinterpret_cast<u32x4_any *>(dst) = b;
                } else {
#pragma unroll
                    for (int z = 0; z < 16; ++z)
                        if (qc + z < rows) dst[z] = (uint8_t)(b[z >> 2] >> (8 * (z & 3)));
                }
            }
            __syncthreads();  // the tile is rewritten by the next one
        }
    }
}

template <typename T, bool VEC>
void quantize(const QuantArgs &a, hipStream_t s) {
    const T *x = static_cast<const T *>(a.x);
    uint8_t *q = static_cast<uint8_t *>(a.q);
    const int64_t most = (int64_t)1 << 22;  // a launch holds fewer than 2^32 threads
    if (a.block_rows == 1 && !a.transpose) {
        // four rows a wave where that still leaves eight waves a SIMD
        const int64_t strips = (a.cols + 511) / 512;
        const bool four = a.rows * strips >= 4 * 8192;
        const int64_t items = (four ? (a.rows + 3) / 4 : a.rows) * strips;
        const dim3 grid((unsigned)std::min((items + 3) / 4, most));
        if (four)
            launch_kernel((quantize_rows_kernel<T, VEC, 4>), grid, dim3(256), s, x, a.rows, a.cols, q, a.scales);
        else
            launch_kernel((quantize_rows_kernel<T, VEC, 1>), grid, dim3(256), s, x, a.rows, a.cols, q, a.scales);
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
//
// A workgroup makes T x T outputs with WN x WM waves, each FN x FM fragments of
// 16 x 16.  Both operands go from global memory straight into LDS, one block of
// 128 along K a stage, while earlier stages are multiplied.  A load instruction
// takes 8 rows x 128 bytes, whole cache lines (16 rows x 64 bytes took 1.63 us
// a stage of 256 + 256 rows without the products, whole lines 1.32).  A stage is
// rows of 128 bytes, the eight pieces of a row XOR-swizzled by the row so that
// fragment reads take distinct banks.  Rows past the matrix and pieces past K
// read as zeros (the buffer's bounds).
//
// What bounds it: a CU's loads into LDS (64 KB a step of 256 x 256 x 128, as
// long as the step's MFMAs) and, at short K, the tile's start and stores.
// Measured: 8192^3 2.63 PFLOP/s to bf16 and 1.40 to fp32 (the image's matrix
// library: 2.64 and, on bf16 operands, 1.35); 32768 x 12800 x 1280 538 to 548 us
// (557); 256 x 12800 x 1280 11.2 us.  Not kept: four waves of 128 x 128 a workgroup
// (3 to 20% slower), workgroups that walk tiles and start the next one before
// storing (8% slower: its first step waits for the stores), results stored
// from the fragments without LDS (3% slower at 32768 x 12800), a start along K
// rotated by workgroup against equal channels of K = 2^n (no change).
typedef __attribute__((address_space(3))) void lds_void_t;

struct Frag {
    u32x4_t half[2];
};

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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0,
                                             (int)min(bytes, (int64_t)0x7FFFFFFF), 0x00020000);
}

// All but this wave's last N loads have landed and its LDS reads are done, then
// the workgroup's barrier: every wave's are.
template <int N>
__device__ __forceinline__ void stage_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// This wave's loads have landed.
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xF << 8));  // vmcnt(0)
    asm volatile("" ::: "memory");
}

constexpr int kXcds = 8;
constexpr uint32_t kPast = 0x80000000u;  // an offset behind every buffer

// First row of b and of a of this workgroup's tile, and its part of K.
// Consecutive workgroups go to the XCDs in turn: each XCD gets a contiguous
// range of (part, tile), all n tiles of kGroup m tiles before the next, so
// that the workgroups of an L2 share operand rows of the same part.
template <int BN, int BM>
__device__ __forceinline__ void tile_origin(const ProductArgs &g, int64_t &n0, int64_t &m0, int &split) {
    constexpr uint32_t kGroup = 4;
    const uint32_t tiles_n = (uint32_t)((g.N + BN - 1) / BN), tiles_m = (uint32_t)((g.M + BM - 1) / BM);
    const uint32_t tiles = tiles_n * tiles_m, all = gridDim.x;
    const uint32_t xq = all / kXcds, xr = all % kXcds, x = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
    const uint32_t logical = x < xr ? x * (xq + 1) + slot : xr * (xq + 1) + (x - xr) * xq + slot;
    split = (int)(logical / tiles);
    const uint32_t tile = logical - (uint32_t)split * tiles;
    const uint32_t grp = tile / (kGroup * tiles_n), in = tile - grp * (kGroup * tiles_n);
    const uint32_t gm = min(kGroup, tiles_m - grp * kGroup);
    n0 = (int64_t)(in / gm) * BN;
    m0 = (int64_t)(grp * kGroup + in % gm) * BM;
}

// A wave's FM x 16 rows (from m0) of FN x 16 values (from n0) as bf16.  They
// pass through LDS (`img`, FM * 16 * FN * 32 bytes of the wave's own), so that a
// store instruction writes whole rows of 32 FN bytes instead of 32-byte pieces
// of 16 rows; the pieces of a row are XOR-swizzled by the row.
template <int FN, int FM>
__device__ __forceinline__ void store_bf16(const ProductArgs &g, const f32x4_t (&acc)[FN][FM], uint8_t *img, int64_t m0,
                                           int64_t n0, int lane) {
    constexpr int kRow = FN * 32, kPieces = FN * 2;
    const int fr = lane & 15;
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int piece = 2 * i + (lane >> 5);
            *reinterpret_cast<u32x2_t *>(img + (j * 16 + fr) * kRow + ((piece ^ fr) & (kPieces - 1)) * 16 +
                                         ((lane >> 4) & 1) * 8) =
                u32x2_t{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
        }
    asm volatile("" ::: "memory");  // (a wave reads what it wrote itself; LDS keeps a wave's order)
    uint16_t *c = static_cast<uint16_t *>(g.c);
    // a result larger than the last-level cache is streamed past the caches,
    // which then keep the operands (32768 x 12800 x 1280: 552 -> 538 us)
    const bool vec = g.N % 8 == 0, past = vec && g.M * g.N * 2 > ((int64_t)256 << 20);
    constexpr int kRowsPer = 64 / kPieces;  // rows of one store instruction
#pragma unroll 4
    for (int r0 = 0; r0 < FM * 16; r0 += kRowsPer) {
        const int r = r0 + lane / kPieces, piece = lane % kPieces;
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(img + r * kRow + ((piece ^ r) & (kPieces - 1)) * 16);
        const int64_t m = m0 + r, n = n0 + piece * 8;
        if (m >= g.M) continue;
        uint16_t *dst = c + m * g.N + n;
        if (n + 8 <= g.N) {
            if (past)
                __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t *>(dst));
            else if (vec)
                *reinterpret_cast<u32x4_t *>(dst) = v;
            else
                *reinterpret_cast<u32x4_any *>(dst) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (n + e < g.N) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// NB = 2: two stages of b and three of a (160 KB of LDS at T = 256: all there
// is; 80 KB at T = 128, two workgroups a CU), so that a's loads have two steps
// to land.  NB = 4: four of each.
template <bool F32, int T, int WN, int WM, int NB>
__global__ __launch_bounds__(64 * WN * WM, 2) void product_kernel(ProductArgs g) {
// (The host pass only needs the launch stub, and drops it where it cannot
// check a device builtin's template-dependent arguments.)
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int W = WN * WM, FN = T / 16 / WN, FM = T / 16 / WM;
    constexpr int kStage = T * 128;       // of one operand
    constexpr int kPerWave = T / 8 / W;   // loads of a wave, operand and stage
    static_assert(T / 8 % W == 0 && (NB == 2 || NB == 4), "stages");
    // (separate arrays: the compiler then knows which of them a fragment read
    // and a load in flight touch, and adds no waits of its own)
    __shared__ __attribute__((aligned(1024))) uint8_t b0[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t a0[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t a1[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t a2[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t a3[NB == 4 ? kStage : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b2[NB == 4 ? kStage : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b3[NB == 4 ? kStage : 16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t n0, m0;
    int split;
    tile_origin<T, T>(g, n0, m0, split);

    const int64_t K = g.K;
    const int kb_all = (int)((K + 127) / 128), pitch = (kb_all + 3) / 4 * 4;
    const int kb_first = split * g.split_blocks, kb_last = min(kb_first + g.split_blocks, kb_all);

    const __amdgpu_buffer_rsrc_t bres = make_rsrc(g.b + n0 * K, min((int64_t)T, g.N - n0) * K);
    const __amdgpu_buffer_rsrc_t ares = make_rsrc(g.a + m0 * K, min((int64_t)T, g.M - m0) * K);
    // (A load's row and piece are its vector offset, which the buffer's bounds
    // cover; the position along K is the scalar one, inside the row by in_k.)
    // lane l of a load fills row l / 8 of its 8-row block, place l % 8; piece c
    // of row r sits at place c ^ (r / 2 % 8): 16 consecutive rows of 128 bytes
    // take the 64 banks once (a wave's blocks are all even or all odd)
    static_assert(W % 2 == 0, "one swizzle for all blocks of a wave");
    const int lr = lane >> 3, lpiece = (lane & 7) ^ (((wave & 1) * 8 + lr) >> 1);
    uint32_t off[kPerWave];  // the same in either operand
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) off[i] = (uint32_t)((wave + W * i) * 8 + lr) * (uint32_t)K + lpiece * 16;
    auto issue = [&](const __amdgpu_buffer_rsrc_t &res, uint8_t *st, int kb) {
        const int k = kb * 128;
        const bool in_k = k + lpiece * 16 < (int)K;
#pragma unroll
        for (int i = 0; i < kPerWave; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_void_t *)(st + (wave + W * i) * 1024), 16,
                                                     in_k ? off[i] : kPast, k, 0, 0);
        // (the scheduler would put the fills off until they are waited for)
        __builtin_amdgcn_sched_barrier(0);
    };

    // scale bytes of two blocks (kb even) for this lane's rows
    const int wn = (wave % WN) * FN, wm = (wave / WN) * FM;  // the wave's first row blocks
    const int bshift = g.b_block_rows == 1 ? 0 : 7, ashift = g.a_block_rows == 1 ? 0 : 7;
    const int64_t brows = ((g.N - 1) >> bshift) + 1, arows = ((g.M - 1) >> ashift) + 1;
    const int64_t bs0 = n0 >> bshift, as0 = m0 >> ashift;
    const __amdgpu_buffer_rsrc_t bsres = make_rsrc(g.b_scales + bs0 * pitch, (brows - bs0) * pitch);
    const __amdgpu_buffer_rsrc_t asres = make_rsrc(g.a_scales + as0 * pitch, (arows - as0) * pitch);
    // (a wave's rows of one side lie in one block of 128, so they share a scale
    // row there; the whole offset is the vector one, which the buffer's bounds
    // cover: rows and blocks past the end read as zero)
    const uint32_t bsoff = (uint32_t)((g.b_block_rows == 1 ? wn * 16 + (lane & 15) : wn / 8) * pitch);
    const uint32_t asoff = (uint32_t)((g.a_block_rows == 1 ? wm * 16 + (lane & 15) : wm / 8) * pitch);
    const int bstep = g.b_block_rows == 1 ? 16 * pitch : 0, astep = g.a_block_rows == 1 ? 16 * pitch : 0;
    static_assert(FN <= 8 && 8 % FN == 0 && FM <= 8 && 8 % FM == 0, "a wave's rows inside one block of 128");
    uint32_t sb[FN], sa[FM];
    auto load_scales = [&](int kb, uint32_t (&b2)[FN], uint32_t (&a2)[FM]) {
        // (opaque, or the sums of all rows are kept in registers across the loop)
        uint32_t bo = bsoff, ao = asoff;
        asm volatile("" : "+v"(bo), "+v"(ao));
#pragma unroll
        for (int i = 0; i < FN; ++i)
            b2[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(bsres, bo + (uint32_t)(i * bstep + kb), 0, 0);
#pragma unroll
        for (int j = 0; j < FM; ++j)
            a2[j] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(asres, ao + (uint32_t)(j * astep + kb), 0, 0);
    };

    f32x4_t acc[FN][FM] = {};
    const int fr = lane & 15;
    // this lane's two pieces of a fragment: rows blk * 16 + fr
    const int fp0 = fr * 128 + ((lane >> 4) ^ (fr >> 1)) * 16, fp1 = fr * 128 + (((lane >> 4) + 4) ^ (fr >> 1)) * 16;
    auto read_half = [&](const uint8_t *st, int blk, int h) {
        return *reinterpret_cast<const u32x4_t *>(st + blk * 2048 + (h == 0 ? fp0 : fp1));
    };
    auto read_frag = [&](const uint8_t *st, int blk) {
        Frag f;
        f.half[0] = read_half(st, blk, 0);
        f.half[1] = read_half(st, blk, 1);
        return f;
    };
    auto compute = [&](const uint8_t *sta, const uint8_t *stb, auto opc) {
        constexpr int OP = decltype(opc)::value;  // which byte of sb and sa
        if constexpr (F32) {
            // half a block at a time: its expanded a side is 8 FM registers
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                bf16x8_t ha[FM][2];
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const u32x4_t w = read_half(sta, wm + j, h);
                    const uint32_t s = (sa[j] >> (8 * OP)) & 0xFFu;
                    ha[j][0] = to_bf16x8(w[0], w[1], s);
                    ha[j][1] = to_bf16x8(w[2], w[3], s);
                }
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    const u32x4_t w = read_half(stb, wn + i, h);
                    const uint32_t s = (sb[i] >> (8 * OP)) & 0xFFu;
                    const bf16x8_t hb[2] = {to_bf16x8(w[0], w[1], s), to_bf16x8(w[2], w[3], s)};
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int j = 0; j < FM; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hb[q], ha[j][q], acc[i][j], 0, 0, 0);
                }
            }
        } else {
            Frag fa[FM];
#pragma unroll
            for (int j = 0; j < FM; ++j) fa[j] = read_frag(sta, wm + j);
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const Frag fb = read_frag(stb, wn + i);
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        e4m3x32(fb), e4m3x32(fa[j]), acc[i][j], 0, 0, OP, (int)sb[i], OP, (int)sa[j]);
            }
        }
    };

    // Each step: this block's loads have landed everywhere (later ones, kAhead
    // a wave, may be in flight) and the stages of the block before are free:
    // fill them, multiply.  (The last fills lie past K, or past this split:
    // never multiplied.)  kb_first is even; a pair's scales are loaded a pair
    // ahead.
    constexpr int kAhead = NB == 2 ? kPerWave : 4 * kPerWave;
    uint32_t sb_next[FN], sa_next[FM];
    load_scales(kb_first, sb, sa);
    issue(bres, b0, kb_first);
    issue(ares, a0, kb_first);
    if constexpr (NB == 4) issue(bres, b1, kb_first + 1);
    issue(ares, a1, kb_first + 1);
    if constexpr (NB == 4) {
        issue(bres, b2, kb_first + 2);
        issue(ares, a2, kb_first + 2);
    }
    int kb = kb_first;
    auto step = [&](const uint8_t *cur_a, const uint8_t *cur_b, uint8_t *fill_a, uint8_t *fill_b, auto opc) {
        stage_barrier<kAhead>();
        if constexpr (decltype(opc)::value == 0) load_scales(kb + 2, sb_next, sa_next);
        issue(bres, fill_b, kb + NB - 1);
        issue(ares, fill_a, kb + (NB == 2 ? 2 : 3));
        compute(cur_a, cur_b, opc);
        if constexpr (decltype(opc)::value == 1) {
#pragma unroll
            for (int i = 0; i < FN; ++i) sb[i] = sb_next[i];
#pragma unroll
            for (int j = 0; j < FM; ++j) sa[j] = sa_next[j];
        }
        return ++kb == kb_last;
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    for (;;) {
        if constexpr (NB == 2) {
            if (step(a0, b0, a2, b1, even)) break;
            if (step(a1, b1, a0, b0, odd)) break;
            if (step(a2, b0, a1, b1, even)) break;
            if (step(a0, b1, a2, b0, odd)) break;
            if (step(a1, b0, a0, b1, even)) break;
            if (step(a2, b1, a1, b0, odd)) break;
        } else {
            if (step(a0, b0, a3, b3, even)) break;
            if (step(a1, b1, a0, b0, odd)) break;
            if (step(a2, b2, a1, b1, even)) break;
            if (step(a3, b3, a2, b2, odd)) break;
        }
    }
    if (g.splits > 1 || F32) {
        // fp32: a lane's four n of one m, 16 bytes (the last fills have to land
        // before the workgroup's LDS is given away)
        wait_loads();
        float *c = g.splits > 1 ? static_cast<float *>(g.ws) + (int64_t)split * g.split_elems : static_cast<float *>(g.c);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + (wm + j) * 16 + (lane & 15);
            if (m >= g.M) continue;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int64_t n = n0 + (wn + i) * 16 + 4 * (lane >> 4);
                float *dst = c + m * g.N + n;
                if (n + 4 <= g.N) {
                    *reinterpret_cast<f32x4_any *>(dst) = acc[i][j];
                } else {
#pragma unroll
                    for (int r = 0; r < 3; ++r)
                        if (n + r < g.N) dst[r] = acc[i][j][r];
                }
            }
        }
        return;
    }
    stage_barrier<0>();  // the last fills have landed and every read is done: the stages are free
    constexpr int kImage = FM * 16 * FN * 32, kImages = kStage / kImage;
    static_assert(kImages * 4 >= W, "the waves' images in four stages");
    uint8_t *const home = wave / kImages == 0 ? b0 : wave / kImages == 1 ? b1 : wave / kImages == 2 ? a0 : a1;
    store_bf16<FN, FM>(g, acc, home + wave % kImages * kImage, m0 + wm * 16, n0 + wn * 16, lane);
#endif
}

// Up to 16 rows of a (decode): 16 x 16 outputs per workgroup, its four waves
// take every fourth block of K, fragments straight from global memory to
// registers (nothing is shared that LDS would save), four blocks of a wave in
// flight at once, and the four sums joined in LDS in order.  Such a product is
// one round trip to memory long: what counts is that all of b is asked for at
// once, by as many workgroups as it has rows of 16.
template <bool F32>
__global__ __launch_bounds__(256) void product_skinny_kernel(ProductArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int PF = 4;
    __shared__ f32x4_t sum_s[3][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tiles = (uint32_t)((g.N + 15) / 16);  // (16 rows of a at most)
    const int split = (int)(blockIdx.x / tiles);
    const int64_t n0 = (int64_t)(blockIdx.x - split * tiles) * 16;
    const int64_t K = g.K;
    const int kb_all = (int)((K + 127) / 128), pitch = (kb_all + 3) / 4 * 4;
    const int kb_first = split * g.split_blocks, kb_last = min(kb_first + g.split_blocks, kb_all);
    const int fr = lane & 15, piece = 16 * (lane >> 4);
    // rows past the end repeat the last one (their results are not stored)
    const int64_t n = min(n0 + fr, g.N - 1), m = min((int64_t)fr, g.M - 1);
    const uint8_t *brow = g.b + n * K + piece, *bsc = g.b_scales + (g.b_block_rows == 1 ? n : n >> 7) * pitch;
    const uint8_t *arow = g.a + m * K + piece, *asc = g.a_scales + (g.a_block_rows == 1 ? m : 0) * pitch;
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int kb = kb_first + wave; kb < kb_last; kb += 4 * PF) {
        Frag fb[PF], fa[PF];
        uint32_t sb[PF], sa[PF];
#pragma unroll
        for (int p = 0; p < PF; ++p) {
            const int k = min(kb + 4 * p, kb_last - 1);  // (past the last: loaded, not used)
            const int64_t o = (int64_t)k * 128;
            const bool in0 = o + piece < K, in1 = o + piece + 64 < K;
            fb[p].half[0] = in0 ? *reinterpret_cast<const u32x4_t *>(brow + o) : zero;
            fb[p].half[1] = in1 ? *reinterpret_cast<const u32x4_t *>(brow + o + 64) : zero;
            fa[p].half[0] = in0 ? *reinterpret_cast<const u32x4_t *>(arow + o) : zero;
            fa[p].half[1] = in1 ? *reinterpret_cast<const u32x4_t *>(arow + o + 64) : zero;
            sb[p] = bsc[k];
            sa[p] = asc[k];
        }
#pragma unroll
        for (int p = 0; p < PF; ++p) {
            if (kb + 4 * p >= kb_last) break;
            if constexpr (F32) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int h = q >> 1, o = 2 * (q & 1);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16x8(fb[p].half[h][o], fb[p].half[h][o + 1], sb[p]),
                                                                  to_bf16x8(fa[p].half[h][o], fa[p].half[h][o + 1], sa[p]),
                                                                  acc, 0, 0, 0);
                }
            } else {
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(e4m3x32(fb[p]), e4m3x32(fa[p]), acc, 0, 0, 0,
                                                                       (int)sb[p], 0, (int)sa[p]);
            }
        }
    }
    if (wave > 0) sum_s[wave - 1][lane] = acc;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < 3; ++w) acc += sum_s[w][lane];
    const int64_t mm = fr, nn = n0 + 4 * (lane >> 4);
    if (mm >= g.M) return;
    if (F32 || g.splits > 1) {
        float *c = g.splits > 1 ? static_cast<float *>(g.ws) + split * g.split_elems : static_cast<float *>(g.c);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (nn + r < g.N) c[mm * g.N + nn + r] = acc[r];
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (nn + r < g.N) static_cast<__bf16 *>(g.c)[mm * g.N + nn + r] = (__bf16)acc[r];
    }
#endif
}

// C = the splits' sums in order, rounded to the result's type.
__global__ __launch_bounds__(256) void product_join_kernel(const float *parts, int32_t splits, int64_t split_elems,
                                                           int64_t n, void *c, bool out_bf16) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
        f32x4_t s = *reinterpret_cast<const f32x4_t *>(parts + i);
        for (int32_t z = 1; z < splits; ++z) s += *reinterpret_cast<const f32x4_t *>(parts + z * split_elems + i);
        if (i + 4 <= n) {
            if (out_bf16)
                *reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(c) + i) =
                    u32x2_t{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
            else
                *reinterpret_cast<f32x4_t *>(static_cast<float *>(c) + i) = s;
        } else {
            for (int r = 0; i + r < n; ++r) {
                if (out_bf16)
                    static_cast<__bf16 *>(c)[i + r] = (__bf16)s[r];
                else
                    static_cast<float *>(c)[i + r] = s[r];
            }
        }
    }
}

// How a product is cut.  256 x 256 tiles where they (or they and parts of K of
// at least eight blocks) come to about one workgroup a CU and neither operand
// has so few rows that half a tile is empty (1 x 129280 x 2560 to fp32: 72 us
// against 118 of 256 x 256, 128 x 129280 x 2560: 104 against 147).  Else 64 x 64
// while those fit the chip at once, two a CU (128 x 2560 x 1280: 5.9 us against
// 10 of 128 x 128, 64 x 25600 x 1280: 9.0 against 10.9), and 128 x 128 beyond
// (1024 x 2560 x 1280: 10.8 against 11.7).  Up to 16 rows of a and 8192 of b go
// to 16 x 16 by four waves (1 x 2560 x 1280: 4.1 us against 5.8 of 64 x 64; 1 x
// 12800 x 1280: 7.6 against 5.7).  K is cut in parts of 16 blocks and more where
// the tiles leave CUs idle (a second launch to join shorter parts costs more
// than it saves: 64 x 2560 x 1280 in two, 5.0 + 2.2 us, whole 5.9).
struct ProductCut {
    int tile;
    int32_t splits, split_blocks;
};

ProductCut cut_of(int64_t M, int64_t N, int64_t K) {
    ProductCut c{};
    auto tiles = [&](int t) { return ((N + t - 1) / t) * ((M + t - 1) / t); };
    const int64_t kb = (K + 127) / 128;
    const int64_t wt = tiles(256), ws = std::max<int64_t>(1, std::min<int64_t>(256 / wt, kb / 8));
    int64_t s = ws;
    if (M <= 16 && N <= 64 * 128) {
        c.tile = 16;
        s = std::min<int64_t>(512 / tiles(16), kb / 16);
    } else if (wt * ws >= 192 && std::min(M, N) > 128) {
        c.tile = 256;
    } else {
        c.tile = tiles(64) > 512 ? 128 : 64;
        s = std::min<int64_t>(256 / tiles(c.tile), kb / 16);
    }
    s = std::max<int64_t>(s, 1);
    int64_t per = (kb + s - 1) / s;
    per += per & 1;  // scales are read two blocks at a time
    c.splits = (int32_t)((kb + per - 1) / per);
    c.split_blocks = (int32_t)per;
    return c;
}

int64_t split_elems_of(int64_t M, int64_t N) { return (M * N + 3) / 4 * 4; }

// The most bytes that a product of at most M, N and K takes, or a little more,
// and never less where one of them grows.  Parts of K come to at most `cap` /
// tiles of them, of `blocks` blocks and more each (as in cut_of), so to at most
// cap * tile^2 sums, and to as many as the largest result in the most parts.
// (128 x 128 tiles are never cut: there are more than 128 of them.)
size_t most_parts(int tile, int64_t cap, int64_t blocks, int64_t M, int64_t N, int64_t kb) {
    const int64_t s = std::min(cap, kb / blocks);
    if (s < 2) return 0;
    return (size_t)std::min(cap * tile * tile, s * split_elems_of(M, N)) * 4;
}

template <bool F32, int T, int WN, int WM, int NB>
void product(const ProductArgs &g, hipStream_t s) {
    const int64_t tiles = ((g.N + T - 1) / T) * ((g.M + T - 1) / T);
    launch_kernel((product_kernel<F32, T, WN, WM, NB>), dim3((unsigned)(tiles * g.splits)), dim3(64 * WN * WM), s,
                  g);
}

template <bool F32>
void product_of(const ProductCut &c, const ProductArgs &g, hipStream_t s) {
    if (c.tile == 256)
        product<F32, 256, 2, 4, 2>(g, s);
    else if (c.tile == 128)
        product<F32, 128, 2, 2, 2>(g, s);
    else if (c.tile == 64)
        product<F32, 64, 2, 2, 4>(g, s);
    else
        launch_kernel(product_skinny_kernel<F32>, dim3((unsigned)((g.N + 15) / 16 * g.splits)), dim3(256),
                      s, g);
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

size_t product_workspace(int64_t M, int64_t N, int64_t K) {
    const ProductCut c = cut_of(M, N, K);
    return c.splits > 1 ? (size_t)c.splits * (size_t)split_elems_of(M, N) * 4 : 0;
}

size_t product_workspace_most(int64_t M, int64_t N, int64_t K) {
    const int64_t kb = (K + 127) / 128, wide = ((M + 255) / 256) * ((N + 255) / 256);
    size_t most = std::max(most_parts(64, 256, 16, M, N, kb),
                           most_parts(16, 512, 16, std::min<int64_t>(M, 16), std::min<int64_t>(N, 64 * 128), kb));
    if (std::min(M, N) > 128 && std::min<int64_t>(256, wide * (kb / 8)) >= 192)
        most = std::max(most, most_parts(256, 256, 8, M, N, kb));
    return most;
}

bool product_fits(int64_t M, int64_t N, int64_t K) {
    // one launch: fewer than 2^32 threads (512 of them a 256 x 256 tile, else 256)
    const ProductCut c = cut_of(M, N, K);
    const int64_t tiles = ((N + c.tile - 1) / c.tile) * ((M + c.tile - 1) / c.tile);
    return tiles * c.splits < ((int64_t)1 << (c.tile == 256 ? 23 : 24));
}

void launch_product(const ProductArgs &a, hipStream_t s) {
    const ProductCut c = cut_of(a.M, a.N, a.K);
    ProductArgs g = a;
    g.splits = c.splits;
    g.split_blocks = c.split_blocks;
    g.split_elems = split_elems_of(a.M, a.N);
    if (a.out_bf16)
        product_of<false>(c, g, s);
    else
        product_of<true>(c, g, s);
    if (c.splits > 1) {
        const int64_t n = a.M * a.N;
        launch_kernel(product_join_kernel, dim3((unsigned)std::min<int64_t>((n + 1023) / 1024, (int64_t)1 << 22)), dim3(256),
                      s, static_cast<const float *>(a.ws), c.splits, g.split_elems, n, a.c, a.out_bf16);
    }
}

}  // namespace engram
