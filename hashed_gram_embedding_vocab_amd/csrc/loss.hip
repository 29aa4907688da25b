// loss.hip -- softmax cross entropy of the output head over the vocabulary, and
// its gradients, with no logits kept.
//
//   x[t][v] = scale <h_t, W_v>,  lse_t = log sum_v exp x[t][v],  loss_t = lse_t - x[t][y_t]
//   P[t][v] = g_t scale (exp(x[t][v] - lse_t) - [v = y_t]):  dh = P W,  dW = P^T h
//
// Tokens whose target lies outside [0, vocab) do not count: their loss, lse and
// dh are zero, their h is not read into dW.  Neither is that of a token whose g_t is 0.
//
// Everything is a product on tiles, C[m][n] = sum_k A[m][k] B[n][k], on the
// matrix instructions with fp32 sums; an operand lies along k (rows of k) or
// across it (rows of m or n, one for each k), so that none is transposed in
// memory:
//   logits   A = h   along,  B = W along   (the tile ends as a maximum and a sum
//                                           of each row, or as a tile of P)
//   dh       A = P   along,  B = W across
//   dW       A = P across,   B = h across
// The forward is one such launch and a join of the rows' maxima and sums.  The
// backward takes the vocabulary in pieces: P of a piece goes to memory in bf16,
// both products read it, and dh's sums go on from piece to piece.  P stays in
// memory for a while because dh and dW need it in tiles of opposite order: made
// again for each of them it would cost a third product more than the two.
//
// Values of 32 bits are held as parts, x = x0 + x1 + x2 (what is left after each
// rounding), and multiplied as the products of the parts down to some weight:
//   forward, fp32 plan   h and W in two fp16 parts of 11 bits, three products
//   backward, fp32 plan  h, W and P in three bf16 parts of 8 bits, six products
//                        (P's values span more than fp16 does)
//   fp32 dW of bf16 h    P in three bf16 parts, three products
//   bf16 results         P in one: a rounding of up to 2^-8 of each value, as the
//                        operand beside it has, which a sum of many averages out; of
//                        few tokens in two
// or, where tokens or vocabulary are few, by the fp32 instructions as they are.
//
// 8192 tokens x 129280 x 2560 in bf16: 5.4 TFLOP forward, 16.3 backward; a library's
// product of 8192^3 runs at 1.40 PFLOP/s here.  Forward 4.1 to 4.3 ms on several cards
// (the product 1.33 PFLOP/s), gradients 13.2 ms (P 1.24, dh 1.26, dW 1.31 PFLOP/s, copy and
// join 0.1 ms).  The matrix units are busy 60 to 70 % of the cycles, at 1.9 GHz, where
// their own power holds the clock.  One token: W's 662 MB in 112 us, 5.9 TB/s.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "engram_internal.h"
#include "loss_cut.h"
#include "stage.h"
#include "vec8.h"

namespace engram {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- operands
// A matrix of rows (of m or n) and columns of k values ("along"), or of rows (one
// for each k) of m or n values ("across"), whole or in blocks of 64 x 64 that
// are each contiguous, with zeros up to whole blocks: then a stage is a few runs of
// 8 KB, and not one line each of as many rows, pages and channels.
struct Operand {
    const void *p;
    int64_t row, row64;      // values from a row to the next, and to the one after 64
    int64_t col64;           // values from a column to the one after 64
    int64_t part, size;      // values from one part to the next, and of a part
};

// Rows of `cols` values.
Operand rows_of(const void *p, int64_t rows, int64_t cols) {
    return Operand{p, cols, kBlock * cols, kBlock, rows * cols, rows * cols};
}
Operand blocks_of(const void *p, int64_t rows, int64_t cols) {
    const int64_t n = round64(rows) * round64(cols);
    return Operand{p, kBlock, round64(cols) * kBlock, kBlock * kBlock, n, n};
}
// Value (r, c) of a matrix in blocks, `row64` as in its Operand.
__device__ __forceinline__ int64_t block_at(int64_t r, int64_t c, int64_t row64) {
    return (r >> 6) * row64 + (c >> 6) * (kBlock * kBlock) + (r & 63) * kBlock + (c & 63);
}

struct GemmArgs {
    Operand a, b;
    int64_t M, N, K;
    int32_t segs;              // products of parts: one after the other along k
    uint32_t a_parts, b_parts; // four bits each: the parts of product z
    int32_t splits, split_steps;  // parts of K, in stages
    int32_t items;             // tiles times splits
    int32_t round;             // an item's stages are a multiple of this
};

// ---------------------------------------------------------------- tiles
// The items (tile, part of K) of a workgroup.  Consecutive workgroups go to the
// XCDs in turn: each XCD gets a contiguous range of (part, tile), all n tiles of
// kGroup m tiles before the next, so that the workgroups of an L2 share operand
// rows of the same part.
template <int TN, int TM>
struct Items {
    static constexpr uint32_t kGroup = 4;
    uint32_t at, end, stride;
    uint32_t tiles_n, tiles_m;
    __device__ __forceinline__ Items(const GemmArgs &g) {
        tiles_n = (uint32_t)((g.N + TN - 1) / TN);
        tiles_m = (uint32_t)((g.M + TM - 1) / TM);
        const uint32_t all = (uint32_t)g.items, x = blockIdx.x % kXcds, q = all / kXcds, r = all % kXcds;
        const uint32_t from = x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q;
        stride = (gridDim.x + kXcds - 1 - x) / kXcds;  // workgroups of this XCD
        at = from + blockIdx.x / kXcds;
        end = from + q + (x < r ? 1u : 0u);
    }
    __device__ __forceinline__ void origin(uint32_t item, int64_t &n0, int64_t &m0, int &split) const {
        const uint32_t tiles = tiles_n * tiles_m;
        split = (int)(item / tiles);
        const uint32_t tile = item - (uint32_t)split * tiles;
        const uint32_t grp = tile / (kGroup * tiles_n), in = tile - grp * (kGroup * tiles_n);
        const uint32_t gm = min(kGroup, tiles_m - grp * kGroup);
        n0 = (int64_t)(in / gm) * TN;
        m0 = (int64_t)(grp * kGroup + in % gm) * TM;
    }
};

// Stages of an item and product of parts: whole rounds of two or four where a
// workgroup takes several items (`round`), the last of them zeros past K.
template <class E>
__device__ __forceinline__ int steps_in(const GemmArgs &g, int split) {
    const int all = (int)((g.K + 128 / (int)sizeof(E) - 1) / (128 / (int)sizeof(E)));
    const int n = min(g.split_steps, all - split * g.split_steps);
    return (n + g.round - 1) & -g.round;
}

// Fills stages of T rows x 128 bytes of k (64 bf16, 32 fp32), one after the other
// through a workgroup's items, with T / 8 loads of 1 KB shared by W waves.
// Along: 8 rows x 128 bytes a load, the eight pieces of 16 bytes of a row
// XOR-swizzled so that the 16 rows that are read at a time lie in distinct banks
// (two rows fill the banks once): piece c of row r at place c ^ (r / 2 % 8), or,
// where a lane's results are to be eight neighbours (PAIRS), where the rows are
// 8 a + b (a, b < 4), at c ^ (r / 2 % 2 + r / 8 % 4 * 2).
// Across: rows of k of T values.  bf16: the 32-byte granules XOR-swizzled by k, so that
// the eight rows that half a wave reads at a time (k % 4 and k / 8 % 2 vary) lie
// in distinct banks.  fp32: the 64-byte ones, by k / 4 (two of four then share
// their banks where a row has two: a tile of 32).
// A leg is the stages of one item and product of parts.  What issue() does after
// its loads is branch-free, so that it is scheduled between multiplications; the
// leg after the present one is worked out in turn(), called between steps at
// least once a leg.
template <class E, int T, int W, bool ACROSS, bool PAIRS, class ItemsT>
struct Feed {
    static constexpr int kStep = 128 / (int)sizeof(E);
    static constexpr int kLoads = T / 8 / W;
    static_assert(T / 8 % W == 0 && W % 4 == 0, "whole loads, one swizzle for all blocks of a wave");
    struct Leg {
        int64_t at, bytes;     // of the next stage in the operand, and from there to the part's end
        int kb, left;          // its number along k, and the leg's stages from there on
    };
    const Operand &o;
    const GemmArgs &g;
    const ItemsT &it;
    const uint32_t parts;
    const bool is_a;
    const int64_t inc;         // bytes from a stage to the next
    uint32_t off[kLoads];
    int lk;                    // along: this lane's k in a stage
    uint32_t item;             // of the leg after
    int seg;
    bool turned;
    Leg now, after;

    __device__ __forceinline__ Feed(const Operand &op, const GemmArgs &ga, uint32_t part_list, bool a_side, int wave,
                                    int lane, const ItemsT &items)
        : o(op), g(ga), it(items), parts(part_list), is_a(a_side),
          // (64 k a stage of bf16; two stages to 64 k of fp32, whose operands are not in blocks)
          inc((sizeof(E) == 2 ? (ACROSS ? op.row64 : op.col64) : (ACROSS ? kStep * op.row : kStep)) * (int64_t)sizeof(E)) {
        if constexpr (!ACROSS) {
            const int lr = lane >> 3;
            const int swz = PAIRS ? ((lr >> 1) & 1) | (wave & 3) << 1 : ((wave & 1) * 8 + lr) >> 1;
            const int piece = (lane & 7) ^ swz;
            lk = piece * (16 / (int)sizeof(E));
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = (wave + W * i) * 8 + lr;
                off[i] = (uint32_t)(((r >> 6) * o.row64 + (r & 63) * o.row + lk) * (int64_t)sizeof(E));
            }
        } else {
            constexpr int kRowBytes = T * (int)sizeof(E), kLanes = kRowBytes / 16;  // lanes of a row of k
            static_assert(sizeof(E) == 2 || T <= 64, "fp32 tiles");
            lk = 0;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int k = (wave + W * i) * (64 / kLanes) + lane / kLanes, place = lane % kLanes;
                int piece;
                if constexpr (sizeof(E) == 2) {
                    const int f = T == 64 ? ((k >> 1) & 1) | ((k >> 3) & 1) << 1 : (k & 3) | ((k >> 3) & 1) << 2;
                    piece = place ^ (f << 1);
                } else {
                    piece = place ^ ((k >> 2) & (T / 16 - 1)) << 2;
                }
                const int col = piece * (16 / (int)sizeof(E));
                off[i] = (uint32_t)(((col >> 6) * o.col64 + (col & 63) + k * o.row) * (int64_t)sizeof(E));
            }
        }
        item = it.at;
        seg = 0;
        now = leg();
        next();
        after = leg();
        turned = false;
    }
    // the leg of `item` and `seg`: no bytes behind the last item
    __device__ __forceinline__ Leg leg() const {
        Leg l{0, 0, 0, 1 << 30};
        if (item < it.end) {
            int64_t n0, m0;
            int split;
            it.origin(item, n0, m0, split);
            const int64_t r0 = is_a ? m0 : n0, part = (int64_t)((parts >> (4 * seg)) & 15u) * o.part;
            l.kb = split * g.split_steps;
            l.left = steps_in<E>(g, split);
            // (kStep divides 64; a tile starts at a multiple of 64, or in the middle of two)
            const int64_t k = (int64_t)l.kb * kStep, r = T < 64 ? r0 & 63 : 0;
            const int64_t at = ACROSS ? (r0 >> 6) * o.col64 + r + (k >> 6) * o.row64 + (k & 63) * o.row
                                      : (r0 >> 6) * o.row64 + r * o.row + (k >> 6) * o.col64 + (k & 63);
            l.at = (part + at) * (int64_t)sizeof(E);
            l.bytes = (o.size - at) * (int64_t)sizeof(E);
        }
        return l;
    }
    __device__ __forceinline__ void next() {
        if (++seg == g.segs) {
            seg = 0;
            item += it.stride;
        }
    }
    __device__ __forceinline__ void turn() {
        if (turned) {
            next();
            after = leg();
            turned = false;
        }
    }
    // the next stage's loads (zeros past the last item's, and past k)
    __device__ __forceinline__ void issue(uint8_t *st, int wave) {
        // (a round's last stages may lie behind the matrix: no bytes, never fewer)
        const int hi = (int)(now.bytes >> 32);
        const uint32_t low = (uint32_t)now.bytes, cut = low < 0x7FFFFFFFu ? low : 0x7FFFFFFFu;
        const int bytes = hi < 0 ? 0 : hi > 0 ? 0x7FFFFFFF : (int)cut;
        const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(static_cast<const char *>(o.p)) + now.at, (short)0, bytes, 0x00020000);
        const bool in = ACROSS || now.kb * kStep + lk < (int)g.K;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_void_t *)(st + (wave + W * i) * 1024), 16,
                                                     in ? off[i] : kPast, 0, 0, 0);
        const bool last = --now.left == 0;
        now.at = last ? after.at : now.at + inc;
        now.bytes = last ? after.bytes : now.bytes - inc;
        now.kb = last ? after.kb : now.kb + 1;
        now.left = last ? after.left : now.left;
        turned = turned || last;
    }
};

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef short v8i16_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;

// This lane's operand of the matrix instructions for half H of a stage: row
// l % 16 of block `blk` of 16 rows; bf16: k = 32 H + 8 (l / 16) .. + 7 of one
// instruction; fp32: k = 16 H + 4 (l / 16) .. + 3, one each of four instructions
// (which k go together does not matter as long as both sides agree).
// PAIRS: rows l / 4 * 8 + l % 4 (+ 4 in the odd block) of the 32 of two blocks.
// Across in bf16: two transposing reads, each of 4 k (the lanes of a group of 16 give
// four values of one k each and get four k of one row).
template <class E, int T, bool ACROSS, bool PAIRS>
struct Reader {
    uint32_t p0, p1;
    __device__ __forceinline__ Reader(int lane) {
        const int fr = lane & 15, g = lane >> 4;
        if constexpr (!ACROSS) {
            const int r = PAIRS ? (fr >> 2) * 8 + (fr & 3) : fr;
            const int swz = PAIRS ? ((fr >> 1) & 1) | (fr >> 2) << 1 : fr >> 1;
            p0 = r * 128 + (g ^ swz) * 16;
            p1 = r * 128 + ((g + 4) ^ swz) * 16;
        } else if constexpr (sizeof(E) == 2) {
            const int q = (lane >> 2) & 3;  // k = 8 g + q (+ 4)
            p0 = (8 * g + q) * (2 * T) + (lane & 3) * 8;
            p1 = T == 64 ? (q >> 1) | (g & 1) << 1 : q | (g & 1) << 2;
        } else {
            p0 = 4 * g * (4 * T) + fr * 4;
            p1 = g & (T / 16 - 1);
        }
    }
    template <int H>
    __device__ __forceinline__ u32x4_t read(const uint8_t *st, int blk) const {
        if constexpr (!ACROSS) {
            const int at = PAIRS ? (blk >> 1) * 4096 + (blk & 1) * 512 : blk * 2048;
            return *reinterpret_cast<const u32x4_t *>(st + at + (H == 0 ? p0 : p1));
        } else if constexpr (sizeof(E) == 2) {
#if defined(__HIP_DEVICE_COMPILE__)
            const uint8_t *at = st + p0 + (blk ^ p1) * 32 + H * 32 * 2 * T;
            const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t *)(at));
            const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t *)(at + 4 * 2 * T));
            return __builtin_bit_cast(u32x4_t, v8i16_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
#else
            return u32x4_t{};
#endif
        } else {
            const uint8_t *at = st + p0 + (blk ^ p1) * 64 + H * 16 * 4 * T;
            u32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint32_t *>(at + e * 4 * T);
            return v;
        }
    }
};

// ---------------------------------------------------------------- what a tile ends as
// A wave's part of a tile: lane l holds C[m][n .. n + 3] of fragment (i, j),
// m = m0 + 16 j + l % 16, n = n0 + 16 i + 4 (l / 16); PAIRS: of fragments 2 p and 2 p + 1
// together the eight n = n0 + 32 p + 8 (l / 16) ...
// kImage: an end that passes through the stages' LDS, so that its workgroup has
// one item; the others' workgroups take items until there are none, and the next
// one's first stages land while a tile ends.

// Rows' maxima and sums of exponentials over the wave's columns, the target's left
// out, and the targets' logits: a nearly certain token's loss is the logarithm of 1
// and a little, which only survives apart from the 1 (store_loss).  That costs 4% of
// 4096 tokens x 32000 x 512 (132 -> 138 us, moves around the branch) and nothing of
// the training case; sums made twice, or in two forms, cost more.
struct LseEnd {
    static constexpr bool kImage = false, kPairs = false, kEarly = true;
    float scale;
    const int32_t *targets;
    float *xt;                 // [n_tok]
    float2 *part;              // [columns / (16 FN)][n_tok]
    int64_t v0;                // the first column's id
    const int32_t *a_unit, *b_unit;  // fp16 operands: the units of their rows (powers of two)
    template <int FM>
    struct Row {
        int32_t id[FM];
    };
    template <int FM>
    __device__ __forceinline__ Row<FM> rows(const GemmArgs &g, int64_t m0, int lane) const {
        Row<FM> r;
#pragma unroll
        for (int j = 0; j < FM; ++j) r.id[j] = targets[min(m0 + 16 * j + (lane & 15), g.M - 1)];
        return r;
    }
    template <class E, int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], const Row<FM> &row, uint8_t *,
                                        int64_t m0, int64_t n0, int, int lane) const {
        const int nl = 4 * (lane >> 4);
        int32_t y[FM];  // the target's column in the wave's, if it has one
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15), at = (int64_t)row.id[j] - v0 - n0;
            y[j] = m < g.M && at >= 0 && at < 16 * FN && n0 + at < g.N ? (int32_t)at : -1;
        }
        if constexpr (std::is_same<E, _Float16>::value) {
            int32_t u[FM];
#pragma unroll
            for (int j = 0; j < FM; ++j) u[j] = a_unit[min(m0 + 16 * j + (lane & 15), g.M - 1)];
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const i32x4_t v = *reinterpret_cast<const i32x4_t *>(b_unit + min(n0 + nl + 16 * i, (g.N - 1) & ~(int64_t)3));
                // (one of the two alone may pass the range of fp32, where the logit does not)
#pragma unroll
                for (int j = 0; j < FM; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_amdgcn_ldexpf(acc[i][j][r], v[r] + u[j]);
                if (i % 2) __builtin_amdgcn_sched_barrier(0);  // (not all units' registers at once)
            }
        }
        float c = scale * kLog2e;
        if (c <= 0.f) {  // (the largest logit is the smallest sum; or all are 0, and NaN are NaN)
            const float f = c < 0.f ? -1.f : 0.f;
            c = c < 0.f ? -c : 1.f;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] *= f;
        }
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            if (!__any(y[j] >= 0)) continue;
            float at_y = 0.f;
            const int32_t mine = y[j] - nl;  // (below 0 without one)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (mine == 16 * i + r) {
                        at_y = acc[i][j][r] * fabsf(scale);
                        acc[i][j][r] = -INFINITY;
                    }
            if (y[j] >= 0 && ((y[j] >> 2) & 3) == (lane >> 4)) xt[m0 + 16 * j + (lane & 15)] = at_y;
        }
        if (n0 + 16 * FN > g.N) {
            const int32_t left = (int32_t)max(g.N - n0, (int64_t)0) - nl;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (16 * i + r >= left)
#pragma unroll
                        for (int j = 0; j < FM; ++j) acc[i][j][r] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < FN; ++i)
                top = fmaxf(fmaxf(fmaxf(top, acc[i][j][0]), fmaxf(acc[i][j][1], acc[i][j][2])), acc[i][j][3]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            // (no finite one: the sum is of NaN, or of nothing)
            const float from = top == -INFINITY ? 0.f : -top * c;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], c, from));
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            const int64_t m = m0 + 16 * j + (lane & 15);
            if (m < g.M && lane < 16)
                part[(v0 + n0) / (16 * FN) * g.M + m] = float2{top == -INFINITY ? top : top * c, sum};
        }
    }
};

// A tile of P, in `parts` parts of bf16 in blocks, or in fp32 rows of ld: zeros
// behind the vocabulary's end and for tokens that do not count.
struct GradEnd {
    static constexpr bool kImage = false, kPairs = true, kEarly = false;
    float scale;
    const Token *token;        // [n_tok]
    void *p;
    int64_t row64, part, ld;   // blocks: as in their Operand, whole columns
    int32_t parts;
    int64_t v0;
    int64_t stack;             // rows from a token's part to its next one; 0: parts apart
    template <int FM>
    struct Row {
        u32x4_t tok[FM];
    };
    template <int FM>
    __device__ __forceinline__ Row<FM> rows(const GemmArgs &g, int64_t m0, int lane) const {
        Row<FM> r;
#pragma unroll
        for (int j = 0; j < FM; ++j)
            r.tok[j] = *reinterpret_cast<const u32x4_t *>(token + min(m0 + 16 * j + (lane & 15), g.M - 1));
        return r;
    }
    template <class E, int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], const Row<FM> &row, uint8_t *,
                                        int64_t m0, int64_t n0, int, int lane) const {
        constexpr bool PAIRS = sizeof(E) == 2;
        // this lane's columns: nl + col(i) + r
        const int64_t nl = n0 + (PAIRS ? 8 : 4) * (lane >> 4);
        auto col = [](int i) { return PAIRS ? (i >> 1) * 32 + (i & 1) * 4 : i * 16; };
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15);
            const u32x4_t &tok = row.tok[j];
            const float l = __uint_as_float(tok[0]), f = m < g.M ? __uint_as_float(tok[1]) : 0.f;
            const int64_t y = (int64_t)(int32_t)tok[2] - v0 - nl;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[i][j][r] = __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], scale, -l) * kLog2e);
            if (__any(y >= 0 && y < 16 * FN)) {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (y == col(i) + r) acc[i][j][r] -= 1.f;
            }
            if (__any(f == 0.f)) {  // (nothing, whatever their logits are)
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = f == 0.f ? 0.f : acc[i][j][r];
            }
#pragma unroll
            for (int i = 0; i < FN; ++i) acc[i][j] *= f;
        }
        if (n0 + 16 * FN > g.N) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (nl + col(i) + r >= g.N)
#pragma unroll
                        for (int j = 0; j < FM; ++j) acc[i][j][r] = 0.f;
        }
        if constexpr (PAIRS) {
            const int64_t all = (stack ? parts : 1) * g.M, whole = (all + kBlock - 1) / kBlock * kBlock;
            for (int q = 0; q < parts; ++q) {
                uint16_t *to = static_cast<uint16_t *>(p) + (stack ? 0 : q * part);
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    // (rows and columns past the last are zeros up to whole blocks)
                    const int64_t mine = m0 + 16 * j + (lane & 15), m = mine + q * stack;
                    if (mine >= (stack ? g.M : whole)) continue;
#pragma unroll
                    for (int i = 0; i < FN; i += 2) {
                        const int64_t n = nl + col(i);
                        if (n >= ld) continue;
                        const f32x4_t &x = acc[i][j], &z = acc[i + 1][j];
                        *reinterpret_cast<u32x4_t *>(to + block_at(m, n, row64)) =
                            u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(z[0], z[1]),
                                    pack_bf16x2(z[2], z[3])};
                    }
                }
                if (q + 1 < parts)
#pragma unroll
                    for (int j = 0; j < FM; ++j)
#pragma unroll
                        for (int i = 0; i < FN; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[i][j][r] -= (float)(__bf16)acc[i][j][r];
            }
            if (stack) {  // (behind the last part's rows fewer than the first 64 of a tile)
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const int64_t m = all + m0 + 16 * j + (lane & 15);
                    if (m >= whole) continue;
#pragma unroll
                    for (int i = 0; i < FN; i += 2) {
                        const int64_t n = nl + col(i);
                        if (n < ld) *reinterpret_cast<u32x4_t *>(static_cast<uint16_t *>(p) + block_at(m, n, row64)) = u32x4_t{};
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int64_t m = m0 + 16 * j + (lane & 15);
                if (m >= g.M) continue;
#pragma unroll
                for (int i = 0; i < FN; ++i)
                    if (nl + col(i) < ld)
                        *reinterpret_cast<f32x4_t *>(static_cast<float *>(p) + m * ld + nl + col(i)) = acc[i][j];
            }
        }
    }
};

// A wave's FM x 16 rows of FN x 16 values as bf16.  They pass through LDS (`img`,
// FM * 16 * FN * 32 bytes of the wave's own), so that a store instruction writes
// whole rows of 32 FN bytes; the pieces of a row are XOR-swizzled by the row.
template <int FN, int FM>
__device__ __forceinline__ void store_rows(const f32x4_t (&acc)[FN][FM], uint8_t *img, uint16_t *c, int64_t ld,
                                           int64_t rows, int64_t cols, int64_t m0, int64_t n0, int lane) {
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
        if (m < rows && n < cols) *reinterpret_cast<u32x4_t *>(c + m * ld + n) = v;  // (rows are whole pieces)
    }
}

// The sums themselves: fp32 (a split's at `split_elems` from the one before), or
// bf16; over what is there or added to it.  WALKS: fp32, by workgroups that take
// several items of few stages.
template <bool WALKS>
struct SumEnd {
    static constexpr bool kImage = !WALKS, kPairs = false, kEarly = false;
    void *c;
    int64_t ld, split_elems;
    bool bf16, accumulate;
    const int32_t *targets;    // given: rows of tokens that do not count are zeros
    int32_t vocab;
    template <int FM>
    struct Row {
        bool counts[FM];
    };
    template <int FM>
    __device__ __forceinline__ Row<FM> rows(const GemmArgs &g, int64_t m0, int lane) const {
        Row<FM> r;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            r.counts[j] = true;
            if (targets) {
                const int32_t id = targets[min(m0 + 16 * j + (lane & 15), g.M - 1)];
                r.counts[j] = id >= 0 && id < vocab;
            }
        }
        return r;
    }
    template <class E, int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], const Row<FM> &row, uint8_t *img,
                                        int64_t m0, int64_t n0, int split, int lane) const {
#pragma unroll
        for (int j = 0; j < FM; ++j)
            if (!row.counts[j])
#pragma unroll
                for (int i = 0; i < FN; ++i) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if constexpr (!WALKS) {
            if (bf16) {
                uint16_t *const out = static_cast<uint16_t *>(c);
                if (accumulate) {  // (to the fp32 sums: what is there and they are rounded once together)
#pragma unroll
                    for (int j = 0; j < FM; ++j) {
                        const int64_t m = m0 + 16 * j + (lane & 15);
                        if (m >= g.M) continue;
#pragma unroll
                        for (int i = 0; i < FN; ++i) {
                            const int64_t n = n0 + 16 * i + 4 * (lane >> 4);
                            if (n >= g.N) continue;
                            const u32x2_t old = *reinterpret_cast<const u32x2_t *>(out + m * ld + n);
                            acc[i][j] += f32x4_t{__uint_as_float(old[0] << 16), __uint_as_float(old[0] & 0xFFFF0000u),
                                                 __uint_as_float(old[1] << 16), __uint_as_float(old[1] & 0xFFFF0000u)};
                        }
                    }
                }
                store_rows<FN, FM>(acc, img, out, ld, g.M, g.N, m0, n0, lane);
                return;
            }
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
// The order the scheduler is to keep: N instructions of a kind (0x20: loads from
// global memory, 0x100: reads of LDS) spread over M matrix instructions.
template <int KIND, int N, int M, int... I>
__device__ __forceinline__ void spread_of(std::integer_sequence<int, I...>) {
    ((__builtin_amdgcn_sched_group_barrier(KIND, 1, 0),
      __builtin_amdgcn_sched_group_barrier(0x8, M * (I + 1) / N - M * I / N, 0)), ...);
}
template <int KIND, int N, int M>
__device__ __forceinline__ void spread() {
    spread_of<KIND, N, M>(std::make_integer_sequence<int, N>{});
}

// A workgroup makes T x T outputs with WN x WM waves, each FN x FM fragments of
// 16 x 16; b's rows are the matrix instruction's A side, so that a lane ends with
// four neighbours of a row of C.  Operands go from global
// memory straight into LDS, 128 bytes of k a stage, while earlier stages are multiplied.
// NB = 2: two stages of b and three of a (160 KB at 256 x 256; 80 KB at 128 x
// 128, two workgroups a CU), so that a's loads have two steps to land.  NB = 4:
// four of each.
//
// A step multiplies the first half of its stage, which the step before has
// read, while it reads the second; then every wave has read this stage and
// the next one has landed (the barrier): it is filled again, and the next
// stage's first half is read while the second is multiplied.  So no multiply
// waits for a read behind a barrier.
template <class E, class End, int T, int WN, int WM, int NB, int NA, bool AX, bool BX>
__global__ __launch_bounds__(64 * WN * WM, 2) void gemm_kernel(GemmArgs g, End end) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int W = WN * WM, FN = T / 16 / WN, FM = T / 16 / WM;
    constexpr int kStage = T * 128;
    constexpr bool PAIRS = End::kPairs && sizeof(E) == 2;
    static_assert(NA == 2 || NA == 3 || NB == 4, "stages");
    static_assert(!PAIRS || !BX, "pairs of rows along k");
    // (separate arrays: the compiler then knows which of them a fragment read
    // and a load in flight touch, and adds no waits of its own)
    __shared__ __attribute__((aligned(1024))) uint8_t b0[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t b1[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t a0[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t a1[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t a2[NA >= 3 ? kStage : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t a3[NA == 4 ? kStage : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b2[NB == 4 ? kStage : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b3[NB == 4 ? kStage : 16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    typedef Items<T, T> ItemsT;
    const ItemsT it(g);
    if (it.at >= it.end) return;  // (all of its waves)
    Feed<E, T, W, AX, false, ItemsT> fa(g.a, g, g.a_parts, true, wave, lane, it);
    Feed<E, T, W, BX, PAIRS, ItemsT> fb(g.b, g, g.b_parts, false, wave, lane, it);
    auto turn = [&] {
        fa.turn();
        fb.turn();
    };
    const Reader<E, T, AX, false> ra(lane);
    const Reader<E, T, BX, PAIRS> rb(lane);
    const int wn = (wave % WN) * FN, wm = (wave / WN) * FM;  // the wave's first row blocks

    // (64 x 64 and less: sums of their own for each half of a stage, in fp32 for each
    // instruction of it, so that long rows round less.  fp16: of the first parts'
    // products, and of the lighter ones.)
    constexpr bool F16 = std::is_same<E, _Float16>::value;
    constexpr int SETS = F16 ? 2 : T > 64 ? 1 : sizeof(E) == 2 ? 2 : 8;
    f32x4_t acc[SETS][FN][FM] = {};
    struct Half {
        u32x4_t a[FM], b[FN];
    };
    auto read = [&](const uint8_t *sta, const uint8_t *stb, Half &h, auto hc) {
        constexpr int H = decltype(hc)::value;
#pragma unroll
        for (int j = 0; j < FM; ++j) h.a[j] = ra.template read<H>(sta, wm + j);
#pragma unroll
        for (int i = 0; i < FN; ++i) h.b[i] = rb.template read<H>(stb, wn + i);
    };
    auto multiply = [&](const Half &h, const Half &hb, int rows_left, auto hc) {
        constexpr int H = decltype(hc)::value;
        if constexpr (sizeof(E) == 2) {
            f32x4_t(&sum)[FN][FM] = acc[SETS > 1 ? H : 0];
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    if constexpr (F16)
                        sum[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, hb.b[i]),
                                                                           __builtin_bit_cast(f16x8_t, h.a[j]), sum[i][j], 0, 0, 0);
                    else
                        sum[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, hb.b[i]),
                                                                            __builtin_bit_cast(bf16x8_t, h.a[j]), sum[i][j], 0, 0, 0);
                }
        } else {
            // (fragments of rows past the last are left out, and stages past K: a few
            // tokens are bound by W's bytes then, and not by products with nothing)
#pragma unroll
            for (int j = 0; j < FM; ++j)
                if (16 * (wm + j) < rows_left)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < FN; ++i)
                            acc[4 * H + e][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __uint_as_float(hb.b[i][e]), __uint_as_float(h.a[j][e]), acc[4 * H + e][i][j], 0, 0, 0);
        }
    };
    // (kAhead loads a wave may be in flight at a step's barrier.  The last fills
    // and reads lie past the last item: zeros, not used.)
    constexpr int kL = T / 8 / W;
    constexpr int kAhead = NB == 4 ? 4 * kL : NA == 3 ? kL : 0;
    constexpr std::integral_constant<int, 0> lo{};
    constexpr std::integral_constant<int, 1> hi{};
    // (a step's fills may end a leg, which turn() has to see before the next one's)
    auto fill = [&](uint8_t *st_b, uint8_t *st_a) {
        fb.issue(st_b, wave);
        fa.issue(st_a, wave);
    };
    fill(b0, a0);
    turn();
    fill(b1, a1);
    turn();
    if constexpr (NB == 4) {
        fill(b2, a2);
        turn();
        fill(b3, a3);
    } else if constexpr (NA == 3) {
        fa.issue(a2, wave);
    }
    turn();
    Half h0, h1;
    int tile_rows = 0, past = 0;  // (fp32) of the tile's rows those of the result; stages past K at an item's end
    stage_barrier<NB == 4 ? 6 * kL : NA * kL>();
    read(a0, b0, h0, lo);
    int left = 0;
    auto step = [&](uint8_t *cur_a, uint8_t *cur_b, const uint8_t *next_a, const uint8_t *next_b)
                    __attribute__((always_inline)) {
        // (256 x 256: the order is set, or the scheduler gathers the reads and fills
        // and the multiplications wait for them: P 1.29 PFLOP/s against 1.20)
        constexpr bool SET = T == 256;
        constexpr int kReads = (AX ? 2 : 1) * FM + (BX ? 2 : 1) * FN, kMul = FM * FN;
        const int rows = sizeof(E) == 4 && left <= past ? 0 : tile_rows;
        read(cur_a, cur_b, h1, hi);
        multiply(h0, h0, rows, lo);
        if constexpr (SET) {
            spread<0x100, kReads, kMul - 8>();
            __builtin_amdgcn_sched_barrier(0);
        }
        stage_barrier<kAhead>();
        if constexpr (SET) __builtin_amdgcn_sched_barrier(0);
        fill(cur_b, cur_a);
        if constexpr (F16) {  // (a stage's halves are the two parts of its k)
            Half h2;
            read(next_a, next_b, h2, lo);
            multiply(h0, h1, rows, hi);
            multiply(h1, h0, rows, hi);
            h0 = h2;
        } else {
            read(next_a, next_b, h0, lo);
            multiply(h1, h1, rows, hi);
        }
        if constexpr (SET) {
            spread<0x20, 2 * kL, 4 * kL>();
            spread<0x100, kReads, kMul - 4 * kL>();
            __builtin_amdgcn_sched_barrier(0);
        }
        return --left == 0;
    };
    for (uint32_t item = it.at; item < it.end; item += it.stride) {
        int64_t n0, m0;
        int split;
        it.origin(item, n0, m0, split);
        left = steps_in<E>(g, split) * g.segs;
        if constexpr (sizeof(E) == 4) {
            tile_rows = (int)min(g.M - m0, (int64_t)T);
            past = left - min(g.split_steps, (int)((g.K + 31) / 32) - split * g.split_steps);
        }
        // (a tile's rows are asked for ahead of its stages, whose waits then cover
        // them: behind them they would wait for the next tile's first stages.  The
        // 256 x 256 tile of P has no registers left for that.)
        constexpr bool EARLY = End::kEarly || T != 256;
        typename End::template Row<FM> row;
        if constexpr (EARLY) row = end.template rows<FM>(g, m0 + wm * 16, lane);
        for (;;) {  // (whole rounds of the stages, or one item; a leg is a round at least)
            if constexpr (NA == 2) {
                step(a0, b0, a1, b1);
                if (step(a1, b1, a0, b0)) break;
                turn();
            } else if constexpr (NB == 2) {
                if (step(a0, b0, a1, b1)) break;
                turn();
                if (step(a1, b1, a2, b0)) break;
                turn();
                if (step(a2, b0, a0, b1)) break;
                turn();
                if (step(a0, b1, a1, b0)) break;
                turn();
                if (step(a1, b0, a2, b1)) break;
                turn();
                if (step(a2, b1, a0, b0)) break;
                turn();
            } else if constexpr (End::kImage) {
                if (step(a0, b0, a1, b1)) break;
                turn();
                if (step(a1, b1, a2, b2)) break;
                turn();
                if (step(a2, b2, a3, b3)) break;
                turn();
                if (step(a3, b3, a0, b0)) break;
                turn();
            } else {
                step(a0, b0, a1, b1);
                step(a1, b1, a2, b2);
                step(a2, b2, a3, b3);
                if (step(a3, b3, a0, b0)) break;
                turn();
            }
        }
        turn();
        if constexpr (End::kImage) stage_barrier<0>();  // the last fills have landed and every read is done: the stages are free
        constexpr int kImage = FM * 16 * FN * 32, kImages = kStage / kImage;
        static_assert(kImages * 4 >= W, "the waves' images in four stages");
        uint8_t *const home = wave / kImages == 0 ? b0 : wave / kImages == 1 ? b1 : wave / kImages == 2 ? a0 : a1;
        if constexpr (!EARLY) row = end.template rows<FM>(g, m0 + wm * 16, lane);
#pragma unroll
        for (int q = SETS / 2; q > 0; q /= 2)
#pragma unroll
            for (int z = 0; z < q; ++z)
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j) acc[z][i][j] += acc[z + q][i][j];
        end.template run<E, FN, FM>(g, acc[0], row, home + wave % kImages * kImage, m0 + wm * 16, n0 + wn * 16, split, lane);
        if constexpr (End::kImage) return;
#pragma unroll
        for (int z = 0; z < SETS; ++z)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[z][i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        read(a0, b0, h0, lo);  // (once more: its registers are free while the tile ends)
    }
    wait_loads();  // (the last fills land before the workgroup's LDS is given away)
#endif
}

// ---------------------------------------------------------------- the rest
// Copies of x [rows][d] for the products: parts in bf16 in blocks, or (T = Out = float,
// one part) whole rows of fp32; with targets, lse, dloss and token given zeros in the
// rows of tokens that do not count or whose factor is 0, and the tokens' constants;
// zeros up to whole blocks.
template <typename T, typename Out, int PARTS>
__global__ __launch_bounds__(256) void parts_kernel(const T *x, int64_t rows, int32_t d, const int32_t *targets,
                                                    int32_t vocab, Out *out, const float *lse, const float *dloss,
                                                    double factor, Token *token, int32_t copies) {
    constexpr bool BLOCKS = sizeof(Out) == 2;
    const int32_t cols = BLOCKS ? (d + kBlock - 1) / kBlock * kBlock : d, units = cols / 8;
    const int64_t all = BLOCKS ? (rows * copies + kBlock - 1) / kBlock * kBlock : rows, n = all * units;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < n; u += (int64_t)gridDim.x * 256) {
        const int64_t to = quotient(u, units), copy = copies > 1 ? min(to / rows, (int64_t)copies - 1) : 0;
        const int64_t r = to - copy * rows;  // (copies of all rows one after the other)
        const int32_t c = (int32_t)(u - to * units) * 8;
        bool counts = r < rows;
        if (targets && counts) {
            const int32_t id = targets[r];
            // (64 bits: the two factors' product may pass fp32's range where the three's does not)
            const float f = (float)((dloss ? (double)dloss[r] : 1.) * factor);
            counts = id >= 0 && id < vocab && f != 0.f;
            if (c == 0 && copy == 0) token[r] = counts ? Token{lse[r], f, id, 0} : Token{0.f, 0.f, -1, 0};
        }
        F8 v = {};
        if (counts && c < d) v = load8(x + r * d + c);
        if constexpr (BLOCKS) {
            const int64_t at = block_at(to, c, (int64_t)cols * kBlock);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                store8(out + q * n * 8 + at, v);
                if (q + 1 < PARTS)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v.v[i] -= (float)(__bf16)v.v[i];
            }
        } else {
            store8(out + r * d + c, v);
        }
    }
}

// Two fp16 parts of x's rows over their units, in blocks, 32 values' first parts and
// then their second ones: a stage of 64 brings what three products of parts need, and
// no part is read twice (517 tokens x 32000 x 1024 181 -> 163 us; tiles of 256 x 256, which
// have no registers for it, were 3 to 6% faster where all CUs are busy, and 10% slower else).
// A row's unit is the power of two over which its largest value lies in [2^14, 2^15),
// so that the parts hold 22 bits of whatever is not below 2^-18 of that, and 2^-40 of it
// otherwise.  One wave a row, of one matrix or behind it of a second one (no rows: none).
struct Halves {
    const float *x;
    int64_t rows, all;         // with those up to whole blocks
    _Float16 *out;
    int32_t *unit;             // exponents
};
__global__ __launch_bounds__(256) void half_parts_kernel(Halves first, Halves second, int32_t d) {
    const int lane = threadIdx.x & 63;
    const int32_t cols = (d + 31) / 32 * 32;
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    for (int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); at < first.all + second.all; at += (int64_t)gridDim.x * 4) {
        const bool one = at < first.all;
        const float *const x = one ? first.x : second.x;
        _Float16 *const out = one ? first.out : second.out;
        int32_t *const unit = one ? first.unit : second.unit;
        const int64_t r = one ? at : at - first.all, rows = one ? first.rows : second.rows;
        uint32_t top = 0u;
        if (r < rows)
            for (int32_t c = lane * 8; c < d; c += 512) {
                const F8 v = load8(x + r * d + c);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t b = __float_as_uint(v.v[i]) & 0x7FFFFFFFu;
                    top = max(top, b < 0x7F800000u ? b : 0u);
                }
            }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
        // exponents of the unit and its inverse, both normal numbers
        const int e = min(max((int)(top >> 23) - 14, 1), 253);
        const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
        if (lane == 0) unit[r] = e - 127;
        for (int32_t c = lane * 8; c < cols; c += 512) {
            F8 v = {};
            if (r < rows && c < d) v = load8(x + r * d + c);
            h8 p0, p1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = v.v[i] * inv;
                p0[i] = (_Float16)y;
                p1[i] = (_Float16)(y - (float)p0[i]);
            }
            _Float16 *to = out + block_at(r, (c >> 5) * 64 + (c & 31), (int64_t)cols * 2 * kBlock);
            *reinterpret_cast<h8 *>(to) = p0;
            *reinterpret_cast<h8 *>(to + 32) = p1;
        }
    }
}

// The largest and the sum of 256 / TB threads' values for each of TB tokens (a
// token's threads lie TB apart); every thread gets them.
template <int TB, bool MAX>
__device__ __forceinline__ float join_threads(float x, float (&red)[256]) {
    red[threadIdx.x] = x;
    __syncthreads();
#pragma unroll
    for (int n = 128; n >= TB; n >>= 1) {
        if ((int)threadIdx.x < n) {
            const float a = red[threadIdx.x], b = red[threadIdx.x + n];
            red[threadIdx.x] = MAX ? fmaxf(a, b) : a + b;
        }
        __syncthreads();
    }
    x = red[threadIdx.x % TB];
    __syncthreads();
    return x;
}

// lse and loss of a token from its target's logit and the others' maximum and sum of
// exponentials, exp(a) of the target's own: loss = log(1 + exp(a)).
__device__ __forceinline__ void store_loss(int64_t t, double top, float sum, int32_t id, int32_t vocab, float x_y,
                                           float *loss, float *lse) {
    const double others = top + (double)logf(sum), a = others - (double)x_y;
    const double f = (double)log1pf(expf(-fabsf((float)a)));  // (of the smaller over the larger)
    const bool counts = id >= 0 && id < vocab;
    loss[t] = counts ? (float)(a > 0. ? a + f : a != a ? a : f) : 0.f;
    lse[t] = counts ? (float)((a > 0. ? others : a != a ? a : (double)x_y) + f) : 0.f;
}

// lse and loss of TB tokens a workgroup from their parts (maxima in powers of two).
// TB = 1, where the parts are many and few workgroups read them, takes the maximum
// first: a thread's loads are then all in flight, with no exponential between them.
template <int TB>
__global__ __launch_bounds__(256) void lse_join_kernel(const float2 *part, int64_t n_parts, int64_t n_tok,
                                                       const int32_t *targets, int32_t vocab, const float *xt, float *loss,
                                                       float *lse) {
    __shared__ float red[256];
    const int64_t t = (int64_t)blockIdx.x * TB + threadIdx.x % TB, tc = min(t, n_tok - 1);
    float top = -INFINITY, sum = 0.f, from;
    if constexpr (TB == 1) {
#pragma unroll 8
        for (int64_t i = threadIdx.x; i < n_parts; i += 256) top = fmaxf(top, part[i * n_tok + tc].x);
        top = join_threads<TB, true>(top, red);
        from = top == -INFINITY ? 0.f : top;
#pragma unroll 8
        for (int64_t i = threadIdx.x; i < n_parts; i += 256) {
            const float2 p = part[i * n_tok + tc];
            sum += p.y * __builtin_amdgcn_exp2f(p.x - from);
        }
    } else {
#pragma unroll 8
        for (int64_t i = threadIdx.x / TB; i < n_parts; i += 256 / TB) {
            const float2 p = part[i * n_tok + tc];
            const float m = fmaxf(top, p.x), f = m == -INFINITY ? 0.f : m;
            sum = sum * __builtin_amdgcn_exp2f(top - f) + p.y * __builtin_amdgcn_exp2f(p.x - f);
            top = m;
        }
        const float own = top;
        top = join_threads<TB, true>(top, red);
        from = top == -INFINITY ? 0.f : top;
        sum *= __builtin_amdgcn_exp2f(own - from);
    }
    sum = join_threads<TB, false>(sum, red);
    if (threadIdx.x < TB && t < n_tok) 
        store_loss(t, top == -INFINITY ? 0. : (double)top * 0.69314718055994530942, sum, targets[t], vocab, xt[t], loss, lse);
}

// From logits in memory (a few tokens of a small vocabulary): the sums of the
// splits of K, in order.
__device__ __forceinline__ float few_logit(const float *x, int64_t at, int32_t splits, int64_t split_elems) {
    float v = x[at];
    for (int32_t z = 1; z < splits; ++z) v += x[z * split_elems + at];
    return v;
}

// One workgroup a token; a thread's logits stay in its registers.
__global__ __launch_bounds__(kFewThreads) void few_loss_kernel(const float *x, int32_t splits, int64_t split_elems,
                                                               int64_t ld, int32_t vocab, float scale,
                                                               const int32_t *targets, float *loss, float *lse) {
    __shared__ float red[2][kFewThreads / 64];
    __shared__ float at_y;
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int32_t id = targets[t];
    float v[kFewEach], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kFewEach; ++i) {
        const int32_t c = i * kFewThreads + (int32_t)threadIdx.x;
        v[i] = c < vocab ? x[t * ld + c] : -INFINITY;
    }
    for (int32_t z = 1; z < splits; ++z)
#pragma unroll
        for (int i = 0; i < kFewEach; ++i) {
            const int32_t c = i * kFewThreads + (int32_t)threadIdx.x;
            if (c < vocab) v[i] += x[z * split_elems + t * ld + c];
        }
#pragma unroll
    for (int i = 0; i < kFewEach; ++i) {
        const int32_t c = i * kFewThreads + (int32_t)threadIdx.x;
        if (c < vocab) v[i] *= scale;
        if (c == id && c < vocab) {
            at_y = v[i];
            v[i] = -INFINITY;
        }
        top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if (lane == 0) red[0][w] = top;
    __syncthreads();
    for (int i = 0; i < kFewThreads / 64; ++i) top = fmaxf(top, red[0][i]);
    const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < kFewEach; ++i) sum += __builtin_amdgcn_exp2f((v[i] - from) * kLog2e);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane == 0) red[1][w] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = red[1][0];
        for (int i = 1; i < kFewThreads / 64; ++i) sum += red[1][i];
        store_loss(t, (double)from, sum, id, vocab, at_y, loss, lse);
    }
}

// P of a few tokens: as GradEnd writes it.
__global__ __launch_bounds__(256) void few_grad_kernel(const float *x, int32_t splits, int64_t split_elems, int64_t ldx,
                                                       int64_t n_tok, int32_t vocab, float scale, const Token *token,
                                                       void *p, int64_t row64, int64_t part, int64_t ld, int32_t parts,
                                                       int64_t stack, bool f32) {
    const int64_t rows = f32 ? n_tok : (n_tok + kBlock - 1) / kBlock * kBlock;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = i / ld, v = i - t * ld;
    if (t >= rows) return;
    float y = 0.f;
    if (t < n_tok && v < vocab) {
        const Token k = token[t];
        y = __builtin_amdgcn_exp2f(fmaf(few_logit(x, t * ldx + v, splits, split_elems), scale, -k.lse) * kLog2e);
        if (v == k.target) y -= 1.f;
        y = k.factor == 0.f ? 0.f : y * k.factor;
    }
    if (f32) {
        static_cast<float *>(p)[t * ld + v] = y;
        return;
    }
    __bf16 *const out = static_cast<__bf16 *>(p);
    const int64_t all = parts * n_tok;
    if (stack && t < (all + kBlock - 1) / kBlock * kBlock - all) out[block_at(all + t, v, row64)] = (__bf16)0.f;
    if (stack && t >= n_tok) return;
    for (int32_t q = 0; q < parts; ++q) {
        out[(stack ? 0 : q * part) + block_at(t + q * stack, v, row64)] = (__bf16)y;
        y -= (float)(__bf16)y;
    }
}

// out[m][i] (+)= sum over the splits, in order, rounded to the output's type;
// rows of tokens that do not count are zeros (targets given).  SHARE threads of a
// workgroup take every SHARE-th split each, where few values come in many splits: the
// time is that of loads one behind the other (64 splits of 2560 values 13 -> 5 us).
template <typename T, int SHARE>
__global__ __launch_bounds__(256) void sum_join_kernel(const float *part, int32_t splits, int64_t split_elems,
                                                       int64_t rows, int32_t d, const int32_t *targets, int32_t vocab,
                                                       T *out, bool accumulate) {
    const int32_t units = d / 8;
    const int64_t n = rows * units;
    constexpr int kUnits = 256 / SHARE;
    const int first = threadIdx.x / kUnits, mine = threadIdx.x % kUnits;
    for (int64_t u0 = (int64_t)blockIdx.x * kUnits; u0 < n; u0 += (int64_t)gridDim.x * kUnits) {
        const int64_t u = u0 + mine;
        F8 v = {};
        if (u < n) {
            if (first < splits) v = load8(part + first * split_elems + u * 8);
#pragma unroll 8
            for (int32_t z = first + SHARE; z < splits; z += SHARE) {  // (eight loads in flight)
                const F8 w = load8(part + z * split_elems + u * 8);
#pragma unroll
                for (int i = 0; i < 8; ++i) v.v[i] += w.v[i];
            }
        }
        if constexpr (SHARE > 1) {
            __shared__ F8 red[SHARE][kUnits];
            __syncthreads();  // (the last units' sums are read)
            red[first][mine] = v;
            __syncthreads();
            if (first > 0) continue;
#pragma unroll
            for (int z = 1; z < SHARE; ++z)
#pragma unroll
                for (int i = 0; i < 8; ++i) v.v[i] += red[z][mine].v[i];
        }
        if (u >= n) continue;
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
template <class E, bool AX, bool BX, class End>
void gemm(GemmArgs g, const End &end, int tile, hipStream_t s) {
    g.items = (int32_t)(ceil_div(g.N, tile) * ceil_div(g.M, tile) * g.splits);
    // one 256 x 256 tile's stages fill a CU's LDS, two of the others fit
    const unsigned most = tile == 256 ? 256 : 512, grid = End::kImage ? (unsigned)g.items : std::min((unsigned)g.items, most);
    constexpr int NA = End::kImage ? 3 : 2;
    constexpr bool SHORT = std::is_same<End, SumEnd<true>>::value;  // few stages an item: two of each do
    constexpr int NS = SHORT ? 2 : 4;
    g.round = End::kImage ? 1 : tile <= 64 ? NS : 2;
    if constexpr (sizeof(E) == 4) {
        if constexpr (!SHORT)
            if (tile == 32) {
                launch_kernel((gemm_kernel<E, End, 32, 2, 2, NS, NS, AX, BX>), dim3(grid), dim3(256), s, g, end);
                return;
            }
        launch_kernel((gemm_kernel<E, End, 64, 2, 2, NS, NS, AX, BX>), dim3(grid), dim3(256), s, g, end);
    } else {
        if constexpr (!SHORT && !std::is_same<E, _Float16>::value)
            if (tile == 256) {
                launch_kernel((gemm_kernel<E, End, 256, 2, 4, 2, NA, AX, BX>), dim3(grid), dim3(512), s, g, end);
                return;
            }
        if (tile == 128)
            launch_kernel((gemm_kernel<E, End, 128, 2, 2, 2, NA, AX, BX>), dim3(grid), dim3(256), s, g, end);
        else
            launch_kernel((gemm_kernel<E, End, 64, 2, 2, NS, NS, AX, BX>), dim3(grid), dim3(256), s, g, end);
    }
}

template <typename T, typename Out, int PARTS>
void make_parts(const void *x, int64_t rows, int32_t d, const LossArgs *a, Out *out, Token *token, hipStream_t s,
                int32_t copies = 1) {
    const int64_t n = sizeof(Out) == 2 ? round64(rows * copies) * (round64(d) / 8) : rows * (d / 8);
    launch_kernel((parts_kernel<T, Out, PARTS>), dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20)), dim3(256), s,
                  static_cast<const T *>(x), rows, d, a ? a->targets : static_cast<const int32_t *>(nullptr),
                  a ? a->vocab : 0, out, a ? static_cast<const float *>(a->lse) : static_cast<const float *>(nullptr),
                  a ? a->dloss : static_cast<const float *>(nullptr), a ? (double)a->dloss_scale * (double)a->scale : 0., token,
                  copies);
}

// A copy in blocks of rows of h or W: a bf16 plan's as they are, an fp32 plan's in
// three parts.
void make_blocks(const LossArgs &a, const void *x, int64_t rows, const LossArgs *mask, uint16_t *out, Token *token,
                 hipStream_t s, int32_t copies = 1) {
    if (a.bf16)
        make_parts<uint16_t, uint16_t, 1>(x, rows, a.d, mask, out, token, s, copies);
    else
        make_parts<float, uint16_t, 3>(x, rows, a.d, mask, out, token, s);
}

// Products of bf16 parts: all pairs whose weight is 2^-16 and more, the lightest first,
// so that only the last one's sums are rounded at their full size.
void parts_of(GemmArgs &g, int a_parts, int b_parts) {
    g.segs = 0;
    g.a_parts = g.b_parts = 0;
    for (int w = 2; w >= 0; --w)
        for (int i = 0; i < a_parts; ++i) {
            const int j = w - i;
            if (j < 0 || j >= b_parts) continue;
            g.a_parts |= (uint32_t)i << (4 * g.segs);
            g.b_parts |= (uint32_t)j << (4 * g.segs);
            ++g.segs;
        }
}

template <class E>
void whole(GemmArgs &g) {
    g.splits = 1;
    g.split_steps = (int32_t)ceil_div(g.K, step_of<E>());
}

// At most n parts of K, for an end whose workgroups take one item each (another's
// item is a whole round of stages, which would run into the next part).
void split_steps(GemmArgs &g, int64_t steps, int64_t n) {
    const int64_t per = ceil_div(steps, n);
    g.split_steps = (int32_t)per;
    g.splits = (int32_t)ceil_div(steps, per);
}

void join_sums(const float *part, int64_t splits, int64_t split_elems, int64_t rows, int32_t d, const int32_t *targets,
               int32_t vocab, bool bf16, void *out, bool accumulate, hipStream_t s) {
    const int64_t units = rows * d / 8;
    const bool share = splits >= 16 && units <= 32768;
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(units, share ? 32 : 256), 1 << 20));
    auto go = [&](auto kernel, auto *to) {
        launch_kernel(kernel, grid, dim3(256), s, part, (int32_t)splits, split_elems, rows, d, targets, vocab, to, accumulate);
    };
    if (bf16)
        go(share ? sum_join_kernel<uint16_t, 8> : sum_join_kernel<uint16_t, 1>, static_cast<uint16_t *>(out));
    else
        go(share ? sum_join_kernel<float, 8> : sum_join_kernel<float, 1>, static_cast<float *>(out));
}

template <class E>
void forward(const LossArgs &a, hipStream_t s) {
    constexpr bool F16 = std::is_same<E, _Float16>::value;
    const LossLayout L = loss_layout(a);
    char *ws = static_cast<char *>(a.ws);
    const int64_t d = a.d, V = a.vocab, T = a.n_tok;
    GemmArgs g{};
    g.M = T;
    g.K = F16 ? (d + 31) / 32 * 64 : d;
    parts_of(g, 1, 1);
    const ForwardCut f = forward_cut<E>(a);
    const bool bh = f.blocks_h, bw = f.blocks_w;
    const int64_t piece = f.piece;
    const Cut few = f.cut;
    uint16_t *h = reinterpret_cast<uint16_t *>(ws + L.h), *w = reinterpret_cast<uint16_t *>(ws + L.w);
    int32_t *h_unit = reinterpret_cast<int32_t *>(ws + L.unit), *w_unit = h_unit + round64(T);
    auto halves = [&](const void *x, int64_t rows, uint16_t *out, int32_t *unit) {
        return Halves{static_cast<const float *>(x), rows, round64(rows), reinterpret_cast<_Float16 *>(out), unit};
    };
    g.N = std::min(piece, V);
    if (bh && !F16) make_blocks(a, a.h, T, nullptr, h, nullptr, s);
    g.a = bh ? blocks_of(h, T, g.K) : rows_of(a.h, T, d);
    if constexpr (!F16) {
        if (few.splits > 1) {
            float *x = reinterpret_cast<float *>(ws + L.few);
            const int64_t ld = round8(V);
            g.b = rows_of(a.w, V, d);
            split_steps(g, ceil_div(d, step_of<E>()), few.splits);
            gemm<E, false, false>(g, SumEnd<false>{x, ld, T * ld, false, false, nullptr, 0}, few.tile, s);
            launch_kernel(few_loss_kernel, dim3((unsigned)T), dim3(kFewThreads), s, x, g.splits, T * ld, ld, a.vocab, a.scale,
                          a.targets, a.loss, a.lse);
            return;
        }
    }
    whole<E>(g);
    LseEnd end{a.scale, a.targets, reinterpret_cast<float *>(ws + L.xt), reinterpret_cast<float2 *>(ws + L.part), 0,
               h_unit, w_unit};
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        g.N = std::min(piece, V - v0);
        end.v0 = v0;
        const char *rows = static_cast<const char *>(a.w) + v0 * d * (a.bf16 ? 2 : 4);
        if constexpr (F16) {  // (and h with the first piece)
            const Halves hh = v0 == 0 ? halves(a.h, T, h, h_unit) : Halves{}, hw = halves(rows, g.N, w, w_unit);
            launch_kernel(half_parts_kernel, dim3((unsigned)std::min<int64_t>((hh.all + hw.all) / 4, 1 << 20)), dim3(256), s,
                          hh, hw, a.d);
        } else if (bw) {
            make_blocks(a, rows, g.N, nullptr, w, nullptr, s);
        }
        g.b = bw ? blocks_of(w, g.N, g.K) : rows_of(rows, g.N, d);
        gemm<E, false, false>(g, end, few.tile, s);
    }
    // (a workgroup a token where its parts are many and tokens are few)
    const int64_t n_parts = 2 * ceil_div(V, few.tile);
    if (T <= 256 && n_parts >= 256)
        launch_kernel(lse_join_kernel<1>, dim3((unsigned)T), dim3(256), s, end.part, n_parts, T, a.targets, a.vocab, end.xt,
                      a.loss, a.lse);
    else
        launch_kernel(lse_join_kernel<8>, dim3((unsigned)ceil_div(T, 8)), dim3(256), s, end.part, n_parts, T, a.targets,
                      a.vocab, end.xt, a.loss, a.lse);
}

template <class E>
void backward(const LossArgs &a, hipStream_t s) {
    constexpr bool F32 = sizeof(E) == 4;
    const LossLayout L = loss_bwd_layout(a);
    char *ws = static_cast<char *>(a.ws);
    const int64_t d = a.d, V = a.vocab, T = a.n_tok;
    const bool parts = !F32 && !a.bf16;
    const bool stack = stacked(a);
    const int hp = parts ? 3 : 1, pp = F32 ? 1 : p_parts(a, stack);
    Token *token = reinterpret_cast<Token *>(ws + L.xt);
    void *h = ws + L.h, *p = ws + L.part;
    uint16_t *wp = reinterpret_cast<uint16_t *>(ws + L.w);
    float *sum = reinterpret_cast<float *>(ws + L.sum), *wsum = reinterpret_cast<float *>(ws + L.wsum);
    const bool bw = parts || (!F32 && blocks_w(a, false));
    if constexpr (F32)
        make_parts<float, float, 1>(a.h, T, a.d, &a, static_cast<float *>(h), token, s);
    else
        make_blocks(a, a.h, T, &a, static_cast<uint16_t *>(h), token, s, stack ? pp : 1);
    const int64_t TP = stack ? pp * T : T;  // rows of P
    const Operand oh = F32 ? rows_of(h, T, d) : blocks_of(h, TP, d);
    int64_t piece = piece_for(V, p_bytes(a));
    if (bw) piece = std::min(piece, piece_for(V, round64(d) * (parts ? 6 : 2)));
    const bool one_piece = piece >= V;
    Cut cut_h{};
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        const int64_t n = std::min(piece, V - v0), ld = round64(n);
        const Operand op = F32 ? rows_of(p, T, ld) : blocks_of(p, TP, n);
        const char *rows = static_cast<const char *>(a.w) + v0 * d * (a.bf16 ? 2 : 4);
        if (bw) make_blocks(a, rows, n, nullptr, wp, nullptr, s);
        const Operand ow = bw ? blocks_of(wp, n, d) : rows_of(rows, n, d);
        GemmArgs g{};
        {  // P
            g.M = T;
            g.N = n;
            g.K = d;
            g.a = oh;
            g.b = ow;
            parts_of(g, hp, hp);
            // (cut as for one part of P, so that where the vocabulary is one piece dh does not
            // go by dW's type; the pieces do, by P's bytes, and with them the order of dh's sums)
            const int out = F32 ? 4 : 2;
            const Cut few = one_piece ? few_cut<E>(a, n, d, g.segs, out) : cut_for<E>(T, n, d, g.segs, 1, out);
            if (few.splits > 1) {
                float *x = reinterpret_cast<float *>(ws + L.few);
                const int64_t ldx = round8(V);
                split_steps(g, ceil_div(d, step_of<E>()), few.splits);
                gemm<E, false, false>(g, SumEnd<false>{x, ldx, T * ldx, false, false, nullptr, 0}, few.tile, s);
                launch_kernel(few_grad_kernel, dim3((unsigned)ceil_div((F32 ? T : round64(T)) * ld, 256)), dim3(256), s, x,
                              g.splits, T * ldx, ldx, T, a.vocab, a.scale, token, p, op.row64, op.part, ld, pp, stack ? T : 0, F32);
            } else {
                whole<E>(g);
                gemm<E, false, false>(g, GradEnd{a.scale, token, p, op.row64, op.part, ld, pp, v0, stack ? T : 0}, few.tile, s);
            }
        }
        if (a.dh) {
            const int64_t M = (stack ? 2 : 1) * T;  // (two parts below each other)
            g.M = M;
            g.N = d;
            g.K = n;
            g.a = op;
            g.b = ow;
            parts_of(g, hp, hp);
            // (the same cut for every piece: its sums go on from one to the next)
            if (v0 == 0)
                cut_h = cut_for<E>(M, d, n, g.segs, std::min(kMostSplits, sum_bytes(M, a.d) / (M * d * 4)), a.bf16 ? 2 : 4);
            split_steps(g, ceil_div(n, step_of<E>()), cut_h.splits);
            if (v0 == 0) cut_h.splits = g.splits;
            if (one_piece && cut_h.splits == 1 && !stack)
                gemm<E, false, true>(g, SumEnd<false>{a.dh, d, 0, a.bf16, false, a.targets, a.vocab}, cut_h.tile, s);
            else
                gemm<E, false, true>(g, SumEnd<false>{sum, d, M * d, false, v0 > 0, nullptr, 0}, cut_h.tile, s);
        }
        if (a.dw) {
            g.M = n;
            g.N = d;
            g.K = TP;
            g.a = op;
            g.b = oh;
            parts_of(g, stack ? 1 : pp, hp);
            const int64_t most = std::min(kMostSplits, weight_sum_bytes(a.vocab, a.d) / (n * d * 4));
            Cut cut = cut_for<E>(n, d, TP, g.segs, most, a.dw_bf16 ? 2 : 4);
            const Cut walk = cut_for<E>(n, d, TP, g.segs, 1, 4, true);
            const bool walks = !a.dw_bf16 && walk.cost < cut.cost;
            if (walks) cut = walk;
            split_steps(g, ceil_div(TP, step_of<E>()), cut.splits);
            char *out = static_cast<char *>(a.dw) + v0 * d * (a.dw_bf16 ? 2 : 4);
            const bool split = g.splits > 1;
            if (walks)
                gemm<E, true, true>(g, SumEnd<true>{out, d, 0, false, a.accumulate, nullptr, 0}, cut.tile, s);
            else
                gemm<E, true, true>(g, SumEnd<false>{split ? static_cast<void *>(wsum) : out, d, n * d, !split && a.dw_bf16,
                                                     !split && a.accumulate, nullptr, 0}, cut.tile, s);
            if (split) join_sums(wsum, g.splits, n * d, n, a.d, nullptr, 0, a.dw_bf16, out, a.accumulate, s);
        }
    }
    if (a.dh && !(one_piece && cut_h.splits == 1 && !stack))  // (a split's two parts of P follow each other)
        join_sums(sum, cut_h.splits * (stack ? 2 : 1), T * d, T, a.d, a.targets, a.vocab, a.bf16, a.dh, false, s);
}

}  // namespace

void launch_loss(const LossArgs &a, hipStream_t s) {
    if (a.bf16)
        forward<uint16_t>(a, s);
    else if (direct32(a, true))
        forward<float>(a, s);
    else
        forward<_Float16>(a, s);
}

void launch_loss_bwd(const LossArgs &a, hipStream_t s) {
    if (!a.bf16 && direct32(a, false))
        backward<float>(a, s);
    else
        backward<uint16_t>(a, s);
}

}  // namespace engram
