// loss.hip -- softmax cross entropy of the output head over the vocabulary, and
// its gradients, with no logits kept.
//
//   x[t][v] = scale <h_t, W_v>,  lse_t = log sum_v exp x[t][v],  loss_t = lse_t - x[t][y_t]
//   P[t][v] = g_t scale (exp(x[t][v] - lse_t) - [v = y_t]):  dh = P W,  dW = P^T h
//
// Tokens whose target lies outside [0, vocab) do not count: their loss, lse and
// dh are zero, their h is not read into dW.
//
// Everything is a product on tiles, C[m][n] = sum_k A[m][k] B[n][k], on the bf16
// matrix instructions with fp32 sums; an operand lies along k (rows of k) or
// across it (rows of m or n, one for each k), so that none is transposed in
// memory:
//   logits   A = h   along,  B = W along   (the tile ends as a maximum and a sum
//                                           of each row, or as a tile of P)
//   dh       A = P   along,  B = W across
//   dW       A = P across,   B = h across
// The forward is one such launch and a join of the rows' maxima and sums.  The
// backward takes the vocabulary in pieces: P of a piece goes to memory in bf16,
// both products read it, and dh's sums go on from piece to piece.
//
// Values of 32 bits are held as parts of 8 bits of mantissa each, x = x0 + x1 +
// x2 (what is left after each rounding to bf16), and multiplied as the products
// of the parts down to 2^-16: six for two values in three parts.  An fp32 plan's
// h, W and P have three parts; P has two where an fp32 dW is made from bf16
// values, and one (a rounding of 2^-9 of each value, as the other operand has)
// where the results are bf16.
#include <algorithm>
#include <type_traits>

#include "engram_internal.h"
#include "stage.h"
#include "vec8.h"

namespace engram {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kStep = 64;  // k of a stage: 128 bytes

// ---------------------------------------------------------------- operands
// rows x k values in bf16, `parts` of them one after the other.
// along: value (row, k) at row * ld + k; across: at k * ld + row.
struct Operand {
    const uint16_t *p;
    int64_t ld;
    int64_t part;   // values from one part to the next
    int64_t rows;   // along: rows; across: values of a k (a multiple of 8)
};

struct GemmArgs {
    Operand a, b;
    int64_t M, N, K;
    int32_t segs;              // products of parts: one after the other along k
    uint32_t a_parts, b_parts; // four bits each: the parts of product z
    int32_t splits, split_steps;  // parts of K, in stages
};

__device__ __forceinline__ int64_t steps_of(int64_t K) { return (K + kStep - 1) / kStep; }

// Fills stages of T rows x 64 k with T / 8 loads of 1 KB, shared by W waves.
// Along: 8 rows x 128 bytes a load, piece c (16 bytes) of row r at place
// c ^ (r / 2 % 8).  Across: 512 / T rows of k of 2 T bytes, their 32-byte
// granules XOR-swizzled by k, so that the eight rows that half a wave reads at a
// time (k % 4 and k / 8 % 2 vary) lie in distinct banks.
template <int T, int W, bool ACROSS>
struct Feed {
    static constexpr int kLoads = T / 8 / W;
    static_assert(T / 8 % W == 0 && W % 2 == 0, "whole loads, one swizzle for all blocks of a wave");
    Operand o;
    int64_t K, first, r0;
    uint32_t off, step_off;
    int lk;             // along: this lane's k in a stage; across: whether its column is inside
    int kb, kb_first, kb_last, seg, segs;
    uint32_t parts;

    __device__ __forceinline__ void init(const Operand &op, int64_t row0, int64_t K_, int wave, int lane, int first_step,
                                         int last_step, int n_segs, uint32_t part_list) {
        o = op;
        K = K_;
        r0 = row0;
        kb = kb_first = first_step;
        kb_last = last_step;
        seg = 0;
        segs = n_segs;
        parts = part_list;
        if constexpr (!ACROSS) {
            const int lr = lane >> 3, piece = (lane & 7) ^ (((wave & 1) * 8 + lr) >> 1);
            off = (uint32_t)(((int64_t)(wave * 8 + lr) * o.ld + piece * 8) * 2);
            step_off = (uint32_t)(W * 8 * o.ld * 2);
            lk = piece * 8;
        } else {
            constexpr int kRows = 512 / T, kLanes = T / 8;  // k rows of a load, lanes of a row
            const int k = wave * kRows + lane / kLanes, place = lane % kLanes;
            const int f = T == 64 ? ((k >> 1) & 1) | ((k >> 3) & 1) << 1 : (k & 3) | ((k >> 3) & 1) << 2;
            static_assert(W * kRows % 16 == 0, "one swizzle for all loads of a lane");
            const int col = ((place >> 1) ^ f) * 16 + (place & 1) * 8;
            off = (uint32_t)(((int64_t)k * o.ld + col) * 2);
            step_off = (uint32_t)((int64_t)W * kRows * o.ld * 2);
            lk = row0 + col < o.rows;
        }
    }
    // the next stage's loads (none past the last)
    __device__ __forceinline__ void issue(uint8_t *st, int wave) {
        const bool live = seg < segs;
        const uint16_t *base = o.p + (int64_t)((parts >> (4 * (live ? seg : 0))) & 15u) * o.part;
        const int64_t k = (int64_t)kb * kStep;
        uint32_t at = off;
        if constexpr (!ACROSS) {
            const __amdgpu_buffer_rsrc_t res = make_rsrc(base + r0 * o.ld, live ? min((int64_t)T, o.rows - r0) * o.ld * 2 : 0);
            const bool in = k + lk < K;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_void_t *)(st + (wave + W * i) * 1024), 16,
                                                         in ? at : kPast, (int)(k * 2), 0, 0);
                at += step_off;
            }
        } else {
            const __amdgpu_buffer_rsrc_t res =
                make_rsrc(base + k * o.ld + r0, live ? (min((int64_t)kStep, K - k) * o.ld - r0) * 2 : 0);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_void_t *)(st + (wave + W * i) * 1024), 16,
                                                         lk ? at : kPast, 0, 0, 0);
                at += step_off;
            }
        }
        // (the scheduler would put the fills off until they are waited for)
        __builtin_amdgcn_sched_barrier(0);
        if (++kb == kb_last) {
            kb = kb_first;
            ++seg;
        }
    }
};

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;

// This lane's operand of the matrix instruction for half H of a stage (k from
// 32 H): row l % 16 of block `blk` of 16 rows, k = 8 (l / 16) .. + 7.
// Across: two transposing reads, each of 4 k (the lanes of a group of 16 give
// four values of one k each and get four k of one row).
template <int T, bool ACROSS>
struct Reader {
    uint32_t p0, p1;
    __device__ __forceinline__ Reader(int lane) {
        if constexpr (!ACROSS) {
            const int fr = lane & 15, g = lane >> 4;
            p0 = fr * 128 + (g ^ (fr >> 1)) * 16;
            p1 = fr * 128 + ((g + 4) ^ (fr >> 1)) * 16;
        } else {
            const int g = lane >> 4, q = (lane >> 2) & 3;  // k = 8 g + q (+ 4)
            p0 = (8 * g + q) * (2 * T) + (lane & 3) * 8;
            p1 = T == 64 ? (q >> 1) | (g & 1) << 1 : q | (g & 1) << 2;
        }
    }
    template <int H>
    __device__ __forceinline__ bf16x8_t read(const uint8_t *st, int blk) const {
        if constexpr (!ACROSS) {
            return *reinterpret_cast<const bf16x8_t *>(st + blk * 2048 + (H == 0 ? p0 : p1));
        } else {
#if defined(__HIP_DEVICE_COMPILE__)
            const uint8_t *at = st + p0 + (blk ^ p1) * 32 + H * 32 * 2 * T;
            const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t *)(at));
            const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t *)(at + 4 * 2 * T));
            typedef short v8i16_t __attribute__((ext_vector_type(8)));
            return __builtin_bit_cast(bf16x8_t, v8i16_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
#else
            return bf16x8_t{};
#endif
        }
    }
};

// First row of b and of a of this workgroup's tile, and its part of K.
// Consecutive workgroups go to the XCDs in turn: each XCD gets a contiguous
// range of (part, tile), all n tiles of kGroup m tiles before the next, so
// that the workgroups of an L2 share operand rows of the same part.
template <int TN, int TM>
__device__ __forceinline__ void tile_of(const GemmArgs &g, int64_t &n0, int64_t &m0, int &split) {
    constexpr uint32_t kGroup = 4;
    const uint32_t tiles_n = (uint32_t)((g.N + TN - 1) / TN), tiles_m = (uint32_t)((g.M + TM - 1) / TM);
    const uint32_t tiles = tiles_n * tiles_m, all = gridDim.x;
    const uint32_t xq = all / kXcds, xr = all % kXcds, x = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
    const uint32_t logical = x < xr ? x * (xq + 1) + slot : xr * (xq + 1) + (x - xr) * xq + slot;
    split = (int)(logical / tiles);
    const uint32_t tile = logical - (uint32_t)split * tiles;
    const uint32_t grp = tile / (kGroup * tiles_n), in = tile - grp * (kGroup * tiles_n);
    const uint32_t gm = min(kGroup, tiles_m - grp * kGroup);
    n0 = (int64_t)(in / gm) * TN;
    m0 = (int64_t)(grp * kGroup + in % gm) * TM;
}

// ---------------------------------------------------------------- what a tile ends as
// A wave's part of a tile: lane l holds C[m][n .. n + 3] of fragment (i, j),
// m = m0 + 16 j + l % 16, n = n0 + 16 i + 4 (l / 16).

// Rows' maxima and sums of exponentials over the wave's columns, and the
// targets' logits.
struct LseEnd {
    float scale;
    const int32_t *targets;
    float *xt;                 // [n_tok]
    float2 *part;              // [columns / (16 FN)][n_tok]
    int64_t v0;                // the first column's id
    template <int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], uint8_t *, int64_t m0, int64_t n0, int,
                                        int lane) const {
        const int64_t nl = n0 + 4 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int i = 0; i < FN; ++i) acc[i][j] *= scale;
        if (n0 + 16 * FN > g.N) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (nl + 16 * i + r >= g.N)
#pragma unroll
                        for (int j = 0; j < FM; ++j) acc[i][j][r] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15);
            const bool in = m < g.M;
            const int64_t y = in ? (int64_t)targets[m] - v0 - n0 : -1;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, acc[i][j][r]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float from = top == -INFINITY ? 0.f : top;
            float sum = 0.f, at_y = 0.f;
            const bool mine = y >= 0 && y < 16 * FN && n0 + y < g.N && ((y >> 2) & 3) == (lane >> 4);
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (y == 16 * i + 4 * (lane >> 4) + r) at_y = acc[i][j][r];
                    sum += __builtin_amdgcn_exp2f((acc[i][j][r] - from) * kLog2e);
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (mine) xt[m] = at_y;
            if (in && lane < 16) part[(v0 + n0) / (16 * FN) * g.M + m] = float2{top, sum};
        }
    }
};

// A wave's FM x 16 rows of FN x 16 values as bf16.  They pass through LDS (`img`,
// FM * 16 * FN * 32 bytes of the wave's own), so that a store instruction writes
// whole rows of 32 FN bytes; the pieces of a row are XOR-swizzled by the row.
template <int FN, int FM>
__device__ __forceinline__ void store_rows(const f32x4_t (&acc)[FN][FM], uint8_t *img, uint16_t *c, int64_t ld,
                                           int64_t rows, int64_t cols, int64_t m0, int64_t n0, int lane, bool accumulate) {
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
    constexpr int kRowsPer = 64 / kPieces;  // rows of one store instruction
#pragma unroll 4
    for (int r0 = 0; r0 < FM * 16; r0 += kRowsPer) {
        const int r = r0 + lane / kPieces, piece = lane % kPieces;
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(img + r * kRow + ((piece ^ r) & (kPieces - 1)) * 16);
        const int64_t m = m0 + r, n = n0 + piece * 8;
        if (m < rows && n < cols) {  // (rows are whole pieces)
            uint16_t *dst = c + m * ld + n;
            if (accumulate) {
                const F8 old = load8(dst);
                F8 x = Raw8<uint16_t>{v}.get();
#pragma unroll
                for (int e = 0; e < 8; ++e) x.v[e] += old.v[e];
                store8(dst, x);
            } else {
                *reinterpret_cast<u32x4_t *>(dst) = v;
            }
        }
    }
    asm volatile("" ::: "memory");
}

// A tile of P, in `parts` parts: zeros behind the vocabulary's end and for tokens
// that do not count.
struct GradEnd {
    float scale, dloss_scale;
    const int32_t *targets;
    const float *lse, *dloss;  // [n_tok]; dloss may be null: ones
    uint16_t *p;               // [parts][n_tok][ld]
    int64_t ld;
    int32_t parts, vocab;
    int64_t v0;
    template <int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], uint8_t *img, int64_t m0, int64_t n0,
                                        int, int lane) const {
        const int64_t nl = n0 + 4 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15);
            const int64_t t = min(m, g.M - 1);
            const int32_t id = targets[t];
            const bool counts = id >= 0 && id < vocab;
            const int64_t y = (int64_t)id - v0 - nl;
            const float l = lse[t], f = (dloss ? dloss[t] : 1.f) * dloss_scale * scale;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float x = __builtin_amdgcn_exp2f((acc[i][j][r] * scale - l) * kLog2e);
                    if (y == 16 * i + r) x -= 1.f;
                    x *= f;
                    acc[i][j][r] = counts && nl + 16 * i + r < g.N ? x : 0.f;
                }
        }
        for (int q = 0; q < parts; ++q) {
            store_rows<FN, FM>(acc, img, p + q * g.M * ld, ld, g.M, ld, m0, n0, lane, false);
            if (q + 1 < parts)
#pragma unroll
                for (int j = 0; j < FM; ++j)
#pragma unroll
                    for (int i = 0; i < FN; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] -= (float)(__bf16)acc[i][j][r];
        }
    }
};

// The sums themselves: fp32 (a split's at `split_elems` from the one before), or
// bf16; over what is there or added to it.
struct SumEnd {
    void *c;
    int64_t ld, split_elems;
    bool bf16, accumulate;
    template <int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], uint8_t *img, int64_t m0, int64_t n0,
                                        int split, int lane) const {
        if (bf16) {
            store_rows<FN, FM>(acc, img, static_cast<uint16_t *>(c), ld, g.M, g.N, m0, n0, lane, accumulate);
            return;
        }
        float *base = static_cast<float *>(c) + split * split_elems;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15);
            if (m >= g.M) continue;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int64_t n = n0 + 16 * i + 4 * (lane >> 4);
                if (n >= g.N) continue;  // (N % 8 == 0)
                f32x4_t *dst = reinterpret_cast<f32x4_t *>(base + m * ld + n);
                *dst = accumulate ? *dst + acc[i][j] : acc[i][j];
            }
        }
    }
};

// ---------------------------------------------------------------- the product
// A workgroup makes TN x TM outputs with WN x WM waves, each FN x FM fragments of
// 16 x 16; b's rows are the matrix instruction's A side.  Operands go from global
// memory straight into LDS, 64 k a stage, while earlier stages are multiplied.
// NB = 2: two stages of b and three of a (160 KB at 256 x 256; 80 KB at 128 x
// 128, two workgroups a CU), so that a's loads have two steps to land.  NB = 4:
// four of each.
template <class End, int TN, int TM, int WN, int WM, int NB, bool AX, bool BX>
__global__ __launch_bounds__(64 * WN * WM, 2) void gemm_kernel(GemmArgs g, End end) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int W = WN * WM, FN = TN / 16 / WN, FM = TM / 16 / WM;
    constexpr int kStageB = TN * 128, kStageA = TM * 128;
    static_assert(TN == TM && (NB == 2 || NB == 4), "stages");
    // (separate arrays: the compiler then knows which of them a fragment read
    // and a load in flight touch, and adds no waits of its own)
    __shared__ __attribute__((aligned(1024))) uint8_t b0[kStageB];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[kStageB];
    __shared__ __attribute__((aligned(1024))) uint8_t a0[kStageA];
    __shared__ __attribute__((aligned(1024))) uint8_t a1[kStageA];
    __shared__ __attribute__((aligned(1024))) uint8_t a2[kStageA];
    __shared__ __attribute__((aligned(1024))) uint8_t a3[NB == 4 ? kStageA : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b2[NB == 4 ? kStageB : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b3[NB == 4 ? kStageB : 16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t n0, m0;
    int split;
    tile_of<TN, TM>(g, n0, m0, split);
    const int all = (int)steps_of(g.K), first = split * g.split_steps, last = min(first + g.split_steps, all);
    Feed<TM, W, AX> fa;
    Feed<TN, W, BX> fb;
    fa.init(g.a, m0, g.K, wave, lane, first, last, g.segs, g.a_parts);
    fb.init(g.b, n0, g.K, wave, lane, first, last, g.segs, g.b_parts);
    const Reader<TM, AX> ra(lane);
    const Reader<TN, BX> rb(lane);
    const int wn = (wave % WN) * FN, wm = (wave / WN) * FM;  // the wave's first row blocks

    f32x4_t acc[FN][FM] = {};
    auto half = [&](const uint8_t *sta, const uint8_t *stb, auto hc) {
        constexpr int H = decltype(hc)::value;
        bf16x8_t va[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j) va[j] = ra.template read<H>(sta, wm + j);
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const bf16x8_t vb = rb.template read<H>(stb, wn + i);
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, va[j], acc[i][j], 0, 0, 0);
        }
    };
    // Each step: this stage's loads have landed everywhere (later ones, kAhead
    // a wave, may be in flight) and the stages of the step before are free:
    // fill them, multiply.  (The last fills lie past the last step: zeros.)
    constexpr int kAhead = NB == 2 ? Feed<TM, W, AX>::kLoads : 2 * (Feed<TM, W, AX>::kLoads + Feed<TN, W, BX>::kLoads);
    fb.issue(b0, wave);
    fa.issue(a0, wave);
    if constexpr (NB == 4) fb.issue(b1, wave);
    fa.issue(a1, wave);
    if constexpr (NB == 4) {
        fb.issue(b2, wave);
        fa.issue(a2, wave);
    }
    int left = (last - first) * g.segs;
    auto step = [&](const uint8_t *cur_a, const uint8_t *cur_b, uint8_t *fill_a, uint8_t *fill_b) {
        stage_barrier<kAhead>();
        fb.issue(fill_b, wave);
        fa.issue(fill_a, wave);
        half(cur_a, cur_b, std::integral_constant<int, 0>{});
        half(cur_a, cur_b, std::integral_constant<int, 1>{});
        return --left == 0;
    };
    for (;;) {
        if constexpr (NB == 2) {
            if (step(a0, b0, a2, b1)) break;
            if (step(a1, b1, a0, b0)) break;
            if (step(a2, b0, a1, b1)) break;
            if (step(a0, b1, a2, b0)) break;
            if (step(a1, b0, a0, b1)) break;
            if (step(a2, b1, a1, b0)) break;
        } else {
            if (step(a0, b0, a3, b3)) break;
            if (step(a1, b1, a0, b0)) break;
            if (step(a2, b2, a1, b1)) break;
            if (step(a3, b3, a2, b2)) break;
        }
    }
    stage_barrier<0>();  // the last fills have landed and every read is done: the stages are free
    constexpr int kImage = FM * 16 * FN * 32, kImages = kStageB / kImage;
    static_assert(kImages * 4 >= W, "the waves' images in four stages");
    uint8_t *const home = wave / kImages == 0 ? b0 : wave / kImages == 1 ? b1 : wave / kImages == 2 ? a0 : a1;
    end.run(g, acc, home + wave % kImages * kImage, m0 + wm * 16, n0 + wn * 16, split, lane);
#endif
}

// ---------------------------------------------------------------- the rest
// Parts of x [rows][d] in bf16, rows of tokens that do not count as zeros
// (targets given): with one part a masked copy.
template <typename T, int PARTS>
__global__ __launch_bounds__(256) void parts_kernel(const T *x, int64_t rows, int32_t d, const int32_t *targets,
                                                    int32_t vocab, uint16_t *out) {
    const int32_t units = d / 8;
    const int64_t n = rows * units;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < n; u += (int64_t)gridDim.x * 256) {
        bool counts = true;
        if (targets) {
            const int32_t id = targets[quotient(u, units)];
            counts = id >= 0 && id < vocab;
        }
        F8 v = {};
        if (counts) v = load8(x + u * 8);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            store8(out + (int64_t)q * n * 8 + u * 8, v);
            if (q + 1 < PARTS)
#pragma unroll
                for (int i = 0; i < 8; ++i) v.v[i] -= (float)(__bf16)v.v[i];
        }
    }
}

// lse and loss of 8 tokens a workgroup, their parts shared by 32 lanes each.
__global__ __launch_bounds__(256) void lse_join_kernel(const float2 *part, int64_t n_parts, int64_t n_tok,
                                                       const int32_t *targets, int32_t vocab, const float *xt, float *loss,
                                                       float *lse) {
    __shared__ float2 red[32][8];
    const int tl = threadIdx.x & 7, sl = threadIdx.x >> 3;
    const int64_t t = (int64_t)blockIdx.x * 8 + tl, tc = min(t, n_tok - 1);
    float top = -INFINITY, sum = 0.f;
    auto add = [&](float2 p) {
        const float m = fmaxf(top, p.x), from = m == -INFINITY ? 0.f : m;
        sum = sum * __builtin_amdgcn_exp2f((top - from) * kLog2e) + p.y * __builtin_amdgcn_exp2f((p.x - from) * kLog2e);
        top = m;
    };
#pragma unroll 4
    for (int64_t i = sl; i < n_parts; i += 32) add(part[i * n_tok + tc]);
    red[sl][tl] = float2{top, sum};
    __syncthreads();
    if (threadIdx.x >= 8 || t >= n_tok) return;
    top = -INFINITY;
    sum = 0.f;
    for (int i = 0; i < 32; ++i) add(red[i][tl]);
    const int32_t id = targets[t];
    const bool counts = id >= 0 && id < vocab;
    const float l = (top == -INFINITY ? 0.f : top) + logf(sum);
    loss[t] = counts ? l - xt[t] : 0.f;
    lse[t] = counts ? l : 0.f;
}

// out[m][i] (+)= sum over the splits, in order, rounded to the output's type;
// rows of tokens that do not count are zeros (targets given).
template <typename T>
__global__ __launch_bounds__(256) void sum_join_kernel(const float *part, int32_t splits, int64_t split_elems,
                                                       int64_t rows, int32_t d, const int32_t *targets, int32_t vocab,
                                                       T *out, bool accumulate) {
    const int32_t units = d / 8;
    const int64_t n = rows * units;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < n; u += (int64_t)gridDim.x * 256) {
        F8 v = load8(part + u * 8);
        for (int32_t z = 1; z < splits; ++z) {
            const F8 w = load8(part + z * split_elems + u * 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) v.v[i] += w.v[i];
        }
        if (targets) {
            const int32_t id = targets[quotient(u, units)];
            if (id < 0 || id >= vocab) v = F8{};
        }
        if (accumulate) {
            const F8 old = load8(out + u * 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) v.v[i] += old.v[i];
        }
        store8(out + u * 8, v);
    }
}

// ---------------------------------------------------------------- host side
// How an M x N product is tiled: 256 x 256 where such tiles come to about one
// workgroup a CU, else 64 x 64 while those fit the chip at once or M is that
// short, and 128 x 128 beyond.
int tile_for(int64_t M, int64_t N) {
    auto tiles = [&](int64_t t) { return ((N + t - 1) / t) * ((M + t - 1) / t); };
    if (M > 128 && tiles(256) >= 192) return 256;
    return M <= 64 || tiles(64) <= 512 ? 64 : 128;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <bool AX, bool BX, class End>
void gemm(const GemmArgs &g, const End &end, int tile, hipStream_t s) {
    const unsigned grid = (unsigned)(ceil_div(g.N, tile) * ceil_div(g.M, tile) * g.splits);
    if (tile == 256)
        launch_kernel((gemm_kernel<End, 256, 256, 2, 4, 2, AX, BX>), dim3(grid), dim3(512), s, g, end);
    else if (tile == 128)
        launch_kernel((gemm_kernel<End, 128, 128, 2, 2, 2, AX, BX>), dim3(grid), dim3(256), s, g, end);
    else
        launch_kernel((gemm_kernel<End, 64, 64, 2, 2, 4, AX, BX>), dim3(grid), dim3(256), s, g, end);
}

template <typename T, int PARTS>
void make_parts(const void *x, int64_t rows, int32_t d, const int32_t *targets, int32_t vocab, uint16_t *out,
                hipStream_t s) {
    const int64_t n = rows * (d / 8);
    launch_kernel((parts_kernel<T, PARTS>), dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20)), dim3(256), s,
                  static_cast<const T *>(x), rows, d, targets, vocab, out);
}

// Products of parts: all pairs whose weight is 2^-16 and more.
void parts_of(GemmArgs &g, int a_parts, int b_parts) {
    g.segs = 0;
    g.a_parts = g.b_parts = 0;
    for (int i = 0; i < a_parts; ++i)
        for (int j = 0; j < b_parts; ++j)
            if (i + j < 3) {
                g.a_parts |= (uint32_t)i << (4 * g.segs);
                g.b_parts |= (uint32_t)j << (4 * g.segs);
                ++g.segs;
            }
}

void whole(GemmArgs &g) {
    g.splits = 1;
    g.split_steps = (int32_t)ceil_div(g.K, kStep);
}

// Parts of K for a product of few tiles: as many as fill the chip's slots (one
// 256 x 256 tile a CU, two of the others) evenly, of at least eight stages.
void split_k(GemmArgs &g, int tile, int64_t most) {
    const int64_t tiles = ceil_div(g.M, tile) * ceil_div(g.N, tile), steps = ceil_div(g.K, kStep);
    const int64_t slots = tile == 256 ? 256 : 512;
    most = std::min<int64_t>({most, steps / 8, tiles >= 4 * slots ? 1 : 4 * slots / tiles});
    int64_t best = 1;
    double best_cost = 1e30;
    for (int64_t s = 1; s <= most; ++s) {
        // rounds of the chip times a tile's stages, and a stage's worth for its start and end
        const double cost = (double)ceil_div(tiles * s, slots) * ((double)ceil_div(steps, s) + 12.);
        if (cost < best_cost * 0.97) {
            best_cost = cost;
            best = s;
        }
    }
    const int64_t per = ceil_div(steps, best);
    g.split_steps = (int32_t)per;
    g.splits = (int32_t)ceil_div(steps, per);
}

constexpr int64_t kPieceBytes = (int64_t)1 << 30;     // of P, and of W's parts, at a time
constexpr int64_t kSumBytes = (int64_t)256 << 20;     // of dh's sums in several splits
constexpr int64_t kMostSplits = 16;

int64_t padded(int64_t vocab) { return ceil_div(vocab, 256) * 256; }

// Columns of the vocabulary taken at a time: `bytes` for each of them may come
// to kPieceBytes, but at least 256 columns.
int64_t piece_for(int64_t vocab, int64_t bytes) {
    const int64_t most = std::max<int64_t>(256, kPieceBytes / bytes / 256 * 256);
    const int64_t n = ceil_div(padded(vocab), most);
    return ceil_div(ceil_div(padded(vocab), n), 256) * 256;
}
// What such a piece takes at most; it never falls as `bytes` grows.
int64_t piece_bytes(int64_t vocab, int64_t bytes) {
    return std::max(256 * bytes, std::min(kPieceBytes, padded(vocab) * bytes));
}

int64_t sum_bytes(int64_t n_tok, int32_t d) {
    const int64_t one = n_tok * d * 4;
    return std::max(one, std::min(kSumBytes, kMostSplits * one));
}

// dW's sums in several splits: at most 64 MB (a tile of each slot).
int64_t weight_sum_bytes(int64_t vocab, int32_t d) { return std::min<int64_t>((int64_t)64 << 20, kMostSplits * vocab * d * 4); }

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// The parts of a token's sums: columns of a wave by the tile's size.  One of the
// largest batch serves the smaller ones (each term grows with the batch, and the
// tiles of 64 and 128 are only taken up to some number of them).
LossLayout loss_layout(const LossArgs &a) {
    LossLayout L{};
    const int64_t v = padded(a.vocab), T = a.n_tok;
    const int64_t n128 = v / 128, n64 = v / 64, n32 = v / 32;
    const int64_t most = std::max({T * n128, std::min<int64_t>(T, 64) * n32, std::min<int64_t>(T * n32, 512 * 128 * 4),
                                   std::min<int64_t>(T, 128) * n64, std::min<int64_t>(T * n64, 192 * 1024 * 4)});
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = off;
        off = round256(off + bytes);
        return (size_t)o;
    };
    L.xt = take(T * 4);
    L.part = take(most * 8);
    if (!a.bf16) {
        L.h = take(3 * T * a.d * 2);
        L.w = take(piece_bytes(a.vocab, (int64_t)a.d * 6));
    }
    L.total = (size_t)off;
    return L;
}

LossLayout loss_bwd_layout(const LossArgs &a) {
    LossLayout L{};
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = off;
        off = round256(off + bytes);
        return (size_t)o;
    };
    const int64_t pp = a.bf16 ? (a.dw_bf16 ? 1 : 2) : 3;
    L.h = take((a.bf16 ? 1 : 3) * a.n_tok * a.d * 2);
    L.part = take(piece_bytes(a.vocab, pp * a.n_tok * 2));
    L.sum = take(sum_bytes(a.n_tok, a.d));
    L.wsum = take(weight_sum_bytes(a.vocab, a.d));
    if (!a.bf16) L.w = take(piece_bytes(a.vocab, (int64_t)a.d * 6));
    L.total = (size_t)off;
    return L;
}

bool loss_fits(int64_t n_tok, int32_t vocab, int32_t d) {
    // tiles of one launch (fewer than 2^32 threads), and 31-bit offsets in a tile's
    // rows of d or of a piece of the vocabulary
    return ceil_div(n_tok, 256) * ceil_div(vocab, 256) < ((int64_t)1 << 22) &&
           ceil_div(n_tok, 256) * ceil_div(d, 256) < ((int64_t)1 << 18) && d <= (1 << 20) && vocab <= (1 << 22) &&
           n_tok <= (1 << 27);
}

void launch_loss(const LossArgs &a, hipStream_t s) {
    const LossLayout L = loss_layout(a);
    char *ws = static_cast<char *>(a.ws);
    LseEnd end{a.scale, a.targets, reinterpret_cast<float *>(ws + L.xt), reinterpret_cast<float2 *>(ws + L.part), 0};
    GemmArgs g{};
    g.M = a.n_tok;
    g.K = a.d;
    whole(g);
    const int64_t d = a.d, V = a.vocab;
    const int64_t piece = a.bf16 ? padded(V) : piece_for(V, d * 6);
    const int tile = tile_for(a.n_tok, std::min(piece, V));
    if (!a.bf16)
        make_parts<float, 3>(a.h, a.n_tok, a.d, nullptr, 0, reinterpret_cast<uint16_t *>(ws + L.h), s);
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        g.N = std::min(piece, V - v0);
        end.v0 = v0;
        if (a.bf16) {
            g.a = Operand{static_cast<const uint16_t *>(a.h), d, 0, a.n_tok};
            g.b = Operand{static_cast<const uint16_t *>(a.w), d, 0, V};
            parts_of(g, 1, 1);
        } else {
            uint16_t *w = reinterpret_cast<uint16_t *>(ws + L.w);
            make_parts<float, 3>(static_cast<const float *>(a.w) + v0 * d, g.N, a.d, nullptr, 0, w, s);
            g.a = Operand{reinterpret_cast<const uint16_t *>(ws + L.h), d, a.n_tok * d, a.n_tok};
            g.b = Operand{w, d, g.N * d, g.N};
            parts_of(g, 3, 3);
        }
        gemm<false, false>(g, end, tile, s);
    }
    const int64_t wave_cols = tile / 2;
    launch_kernel(lse_join_kernel, dim3((unsigned)ceil_div(a.n_tok, 8)), dim3(256), s, end.part,
                  ceil_div(V, tile) * (tile / wave_cols), a.n_tok, a.targets, a.vocab, end.xt, a.loss, a.lse);
}

void launch_loss_bwd(const LossArgs &a, hipStream_t s) {
    const LossLayout L = loss_bwd_layout(a);
    char *ws = static_cast<char *>(a.ws);
    const int64_t d = a.d, V = a.vocab, T = a.n_tok;
    const int hp = a.bf16 ? 1 : 3, pp = a.bf16 ? (a.dw_bf16 ? 1 : 2) : 3;
    uint16_t *h = reinterpret_cast<uint16_t *>(ws + L.h), *p = reinterpret_cast<uint16_t *>(ws + L.part);
    uint16_t *wp = reinterpret_cast<uint16_t *>(ws + L.w);
    float *sum = reinterpret_cast<float *>(ws + L.sum), *wsum = reinterpret_cast<float *>(ws + L.wsum);
    if (a.bf16)
        make_parts<uint16_t, 1>(a.h, T, a.d, a.targets, a.vocab, h, s);
    else
        make_parts<float, 3>(a.h, T, a.d, a.targets, a.vocab, h, s);
    int64_t piece = piece_for(V, (int64_t)pp * T * 2);
    if (!a.bf16) piece = std::min(piece, piece_for(V, d * 6));
    int32_t dh_splits = 1;
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        const int64_t n = std::min(piece, V - v0), ld = ceil_div(n, kStep) * kStep;
        const Operand ph{p, ld, T * ld, T}, pw{p, ld, T * ld, ld};
        Operand w{static_cast<const uint16_t *>(a.w) + v0 * d, d, 0, n};
        if (!a.bf16) {
            make_parts<float, 3>(static_cast<const float *>(a.w) + v0 * d, n, a.d, nullptr, 0, wp, s);
            w = Operand{wp, d, n * d, n};
        }
        GemmArgs g{};
        {  // P
            g.M = T;
            g.N = n;
            g.K = d;
            g.a = Operand{h, d, T * d, T};
            g.b = w;
            whole(g);
            parts_of(g, hp, hp);
            const GradEnd end{a.scale, a.dloss_scale, a.targets, a.lse, a.dloss, p, ld, pp, a.vocab, v0};
            gemm<false, false>(g, end, tile_for(T, n), s);
        }
        if (a.dh) {
            g.M = T;
            g.N = d;
            g.K = n;
            g.a = ph;
            g.b = w;
            g.b.rows = d;
            parts_of(g, a.bf16 ? 1 : 3, hp);
            const int tile = tile_for(T, d);
            // (the same split for every piece: its sums go on from one to the next)
            if (v0 == 0) {
                split_k(g, tile, std::min(kMostSplits, sum_bytes(T, a.d) / (T * d * 4)));
                dh_splits = g.splits;
            } else {
                const int64_t steps = ceil_div(n, kStep);
                g.splits = dh_splits;
                g.split_steps = (int32_t)ceil_div(steps, dh_splits);
                g.splits = (int32_t)ceil_div(steps, g.split_steps);
            }
            const SumEnd end{sum, d, T * d, false, v0 > 0};
            gemm<false, true>(g, end, tile, s);
        }
        if (a.dw) {
            g.M = n;
            g.N = d;
            g.K = T;
            g.a = pw;
            g.b = Operand{h, d, T * d, d};
            parts_of(g, pp, hp);
            const int tile = tile_for(n, d);
            split_k(g, tile, std::min(kMostSplits, weight_sum_bytes(a.vocab, a.d) / (n * d * 4)));
            char *out = static_cast<char *>(a.dw) + v0 * d * (a.dw_bf16 ? 2 : 4);
            const bool parts = g.splits > 1;
            const SumEnd end{parts ? static_cast<void *>(wsum) : out, d, n * d, !parts && a.dw_bf16, !parts && a.accumulate};
            gemm<true, true>(g, end, tile, s);
            if (parts) {
                const dim3 grid((unsigned)std::min<int64_t>((n * d / 8 + 255) / 256, 1 << 20));
                if (a.dw_bf16)
                    launch_kernel(sum_join_kernel<uint16_t>, grid, dim3(256), s, wsum, g.splits, n * d, n, a.d,
                                  static_cast<const int32_t *>(nullptr), 0, reinterpret_cast<uint16_t *>(out),
                                  a.accumulate);
                else
                    launch_kernel(sum_join_kernel<float>, grid, dim3(256), s, wsum, g.splits, n * d, n, a.d,
                                  static_cast<const int32_t *>(nullptr), 0, reinterpret_cast<float *>(out), a.accumulate);
            }
        }
    }
    if (a.dh) {
        const dim3 grid((unsigned)std::min<int64_t>((T * d / 8 + 255) / 256, 1 << 20));
        if (a.bf16)
            launch_kernel(sum_join_kernel<uint16_t>, grid, dim3(256), s, sum, dh_splits, T * d, T, a.d, a.targets,
                          a.vocab, static_cast<uint16_t *>(a.dh), false);
        else
            launch_kernel(sum_join_kernel<float>, grid, dim3(256), s, sum, dh_splits, T * d, T, a.d, a.targets, a.vocab,
                          static_cast<float *>(a.dh), false);
    }
}

}  // namespace engram
