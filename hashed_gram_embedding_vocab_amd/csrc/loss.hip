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
#include <utility>

#include "engram_internal.h"
#include "stage.h"
#include "vec8.h"

namespace engram {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBlock = 64;  // rows and columns of a block of the workspaces' matrices

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
int64_t round64(int64_t x) { return (x + kBlock - 1) / kBlock * kBlock; }
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
// in distinct banks.  fp32: the 64-byte ones, by k / 4 % 4.
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
            static_assert(sizeof(E) == 2 || T == 64, "fp32 tiles");
            lk = 0;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int k = (wave + W * i) * (64 / kLanes) + lane / kLanes, place = lane % kLanes;
                int piece;
                if constexpr (sizeof(E) == 2) {
                    const int f = T == 64 ? ((k >> 1) & 1) | ((k >> 3) & 1) << 1 : (k & 3) | ((k >> 3) & 1) << 2;
                    piece = place ^ (f << 1);
                } else {
                    piece = place ^ ((k >> 2) & 3) << 2;
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
            // (kStep divides 64, and a tile starts at a multiple of 64)
            const int64_t k = (int64_t)l.kb * kStep;
            const int64_t at = ACROSS ? (r0 >> 6) * o.col64 + (k >> 6) * o.row64 + (k & 63) * o.row
                                      : (r0 >> 6) * o.row64 + (k >> 6) * o.col64 + (k & 63);
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
            p1 = g;
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

// Rows' maxima and sums of exponentials over the wave's columns, and the
// targets' logits.
struct LseEnd {
    static constexpr bool kImage = false, kPairs = false;
    float scale;
    const int32_t *targets;
    float *xt;                 // [n_tok]
    float2 *part;              // [columns / (16 FN)][n_tok]
    int64_t v0;                // the first column's id
    template <class E, int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], uint8_t *, int64_t m0, int64_t n0, int,
                                        int lane) const {
        const int nl = 4 * (lane >> 4);
        int32_t y[FM];  // the target's column in the wave's, if it has one
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15), at = (int64_t)targets[min(m, g.M - 1)] - v0 - n0;
            y[j] = m < g.M && at >= 0 && at < 16 * FN && n0 + at < g.N ? (int32_t)at : -1;
        }
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            if (!__any(y[j] >= 0)) continue;
            float at_y = 0.f;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (y[j] == 16 * i + nl + r) at_y = acc[i][j][r] * scale;
            if (y[j] >= 0 && ((y[j] >> 2) & 3) == (lane >> 4)) xt[m0 + 16 * j + (lane & 15)] = at_y;
        }
        float c = scale * kLog2e;
        if (c < 0.f) {  // (the largest logit is the smallest sum)
            c = -c;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] = -acc[i][j];
        }
        if (n0 + 16 * FN > g.N) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n0 + nl + 16 * i + r >= g.N)
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

// What the gradient of a token's logits needs: lse, the factor g_t scale (0 for a
// token that does not count) and the target.
struct Token {
    float lse, factor;
    int32_t target, unused;
};

// A tile of P, in `parts` parts of bf16 in blocks, or in fp32 rows of ld: zeros
// behind the vocabulary's end and for tokens that do not count.
struct GradEnd {
    static constexpr bool kImage = false, kPairs = true;
    float scale;
    const Token *token;        // [n_tok]
    void *p;
    int64_t row64, part, ld;   // blocks: as in their Operand, whole columns
    int32_t parts;
    int64_t v0;
    template <class E, int FN, int FM>
    __device__ __forceinline__ void run(const GemmArgs &g, f32x4_t (&acc)[FN][FM], uint8_t *, int64_t m0, int64_t n0,
                                        int, int lane) const {
        constexpr bool PAIRS = sizeof(E) == 2;
        // this lane's columns: nl + col(i) + r
        const int64_t nl = n0 + (PAIRS ? 8 : 4) * (lane >> 4);
        auto col = [](int i) { return PAIRS ? (i >> 1) * 32 + (i & 1) * 4 : i * 16; };
        u32x4_t tok[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j)
            tok[j] = *reinterpret_cast<const u32x4_t *>(token + min(m0 + 16 * j + (lane & 15), g.M - 1));
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + 16 * j + (lane & 15);
            const float l = __uint_as_float(tok[j][0]), f = m < g.M ? __uint_as_float(tok[j][1]) : 0.f;
            const int64_t y = (int64_t)(int32_t)tok[j][2] - v0 - nl;
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
            for (int q = 0; q < parts; ++q) {
                uint16_t *to = static_cast<uint16_t *>(p) + q * part;
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    // (rows and columns past the last are zeros up to whole blocks)
                    const int64_t m = m0 + 16 * j + (lane & 15);
                    if (m >= (g.M + kBlock - 1) / kBlock * kBlock) continue;
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
}

// The sums themselves: fp32 (a split's at `split_elems` from the one before), or
// bf16; over what is there or added to it.
struct SumEnd {
    static constexpr bool kImage = true, kPairs = false;
    void *c;
    int64_t ld, split_elems;
    bool bf16, accumulate;
    template <class E, int FN, int FM>
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
// 16 x 16; b's rows are the matrix instruction's A side.  Operands go from global
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

    f32x4_t acc[FN][FM] = {};
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
    auto multiply = [&](const Half &h) {
        if constexpr (sizeof(E) == 2) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, h.b[i]),
                                                                        __builtin_bit_cast(bf16x8_t, h.a[j]), acc[i][j], 0, 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(h.b[i][e]), __uint_as_float(h.a[j][e]),
                                                                         acc[i][j], 0, 0, 0);
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
    stage_barrier<NB == 4 ? 6 * kL : NA * kL>();
    read(a0, b0, h0, lo);
    int left = 0;
    auto step = [&](uint8_t *cur_a, uint8_t *cur_b, const uint8_t *next_a, const uint8_t *next_b)
                    __attribute__((always_inline)) {
        // (256 x 256: the order is set, or the scheduler gathers the reads and fills
        // and the multiplications wait for them: P 1.29 PFLOP/s against 1.20)
        constexpr bool SET = T == 256;
        constexpr int kReads = (AX ? 2 : 1) * FM + (BX ? 2 : 1) * FN, kMul = FM * FN;
        read(cur_a, cur_b, h1, hi);
        multiply(h0);
        if constexpr (SET) {
            spread<0x100, kReads, kMul - 8>();
            __builtin_amdgcn_sched_barrier(0);
        }
        stage_barrier<kAhead>();
        if constexpr (SET) __builtin_amdgcn_sched_barrier(0);
        fill(cur_b, cur_a);
        read(next_a, next_b, h0, lo);
        multiply(h1);
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
        end.template run<E, FN, FM>(g, acc, home + wave % kImages * kImage, m0 + wm * 16, n0 + wn * 16, split, lane);
        if constexpr (End::kImage) return;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        read(a0, b0, h0, lo);  // (once more: its registers are free while the tile ends)
    }
    wait_loads();  // (the last fills land before the workgroup's LDS is given away)
#endif
}

// ---------------------------------------------------------------- the rest
// Copies of x [rows][d] for the products: parts in bf16 in blocks, or (T = Out = float,
// one part) whole rows of fp32; zeros in the rows of tokens that do not count
// (targets given) and up to whole blocks.  Beside it the tokens' constants.
template <typename T, typename Out, int PARTS>
__global__ __launch_bounds__(256) void parts_kernel(const T *x, int64_t rows, int32_t d, const int32_t *targets,
                                                    int32_t vocab, Out *out, const float *lse, const float *dloss,
                                                    float factor, Token *token) {
    constexpr bool BLOCKS = sizeof(Out) == 2;
    const int32_t cols = BLOCKS ? (d + kBlock - 1) / kBlock * kBlock : d, units = cols / 8;
    const int64_t all = BLOCKS ? (rows + kBlock - 1) / kBlock * kBlock : rows, n = all * units;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < n; u += (int64_t)gridDim.x * 256) {
        const int64_t r = quotient(u, units);
        const int32_t c = (int32_t)(u - r * units) * 8;
        bool counts = r < rows;
        if (targets && counts) {
            const int32_t id = targets[r];
            counts = id >= 0 && id < vocab;
            if (token && c == 0)
                token[r] = Token{lse[r], counts ? (dloss ? dloss[r] : 1.f) * factor : 0.f, id, 0};
        }
        F8 v = {};
        if (counts && c < d) v = load8(x + r * d + c);
        if constexpr (BLOCKS) {
            const int64_t at = block_at(r, c, (int64_t)cols * kBlock);
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

// lse and loss of 8 tokens a workgroup, their parts (maxima in powers of two)
// shared by 32 lanes each.
__global__ __launch_bounds__(256) void lse_join_kernel(const float2 *part, int64_t n_parts, int64_t n_tok,
                                                       const int32_t *targets, int32_t vocab, const float *xt, float *loss,
                                                       float *lse) {
    __shared__ float2 red[32][8];
    const int tl = threadIdx.x & 7, sl = threadIdx.x >> 3;
    const int64_t t = (int64_t)blockIdx.x * 8 + tl, tc = min(t, n_tok - 1);
    float top = -INFINITY, sum = 0.f;
    auto add = [&](float2 p) {
        const float m = fmaxf(top, p.x), from = m == -INFINITY ? 0.f : m;
        sum = sum * __builtin_amdgcn_exp2f(top - from) + p.y * __builtin_amdgcn_exp2f(p.x - from);
        top = m;
    };
#pragma unroll 8
    for (int64_t i = sl; i < n_parts; i += 32) add(part[i * n_tok + tc]);
    red[sl][tl] = float2{top, sum};
    __syncthreads();
    if (threadIdx.x >= 8 || t >= n_tok) return;
    top = -INFINITY;
    sum = 0.f;
    for (int i = 0; i < 32; ++i) add(red[i][tl]);
    const int32_t id = targets[t];
    const bool counts = id >= 0 && id < vocab;
    const float l = (float)((top == -INFINITY ? 0. : (double)top * 0.69314718055994530942) + (double)logf(sum));
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
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class E>
constexpr int64_t step_of() {
    return 128 / (int64_t)sizeof(E);
}

// How an M x N product is tiled: 256 x 256 where such tiles (or they and parts of
// K of at least eight stages, where K may be split) come to about one workgroup
// a CU, else 64 x 64 while those fit the chip at once or M is that short, and
// 128 x 128 beyond.  fp32 tiles are 64 x 64.
int tile_for(int64_t M, int64_t N, int64_t k_steps = 0) {
    auto tiles = [&](int64_t t) { return ((N + t - 1) / t) * ((M + t - 1) / t); };
    const int64_t wide = tiles(256), parts = std::max<int64_t>(1, std::min<int64_t>(256 / wide, k_steps / 8));
    if (std::min(M, k_steps ? N : M) > 128 && wide * parts >= 192) return 256;
    return M <= 64 || tiles(64) <= 512 ? 64 : 128;
}

template <class E, bool AX, bool BX, class End>
void gemm(GemmArgs g, const End &end, int tile, hipStream_t s) {
    g.items = (int32_t)(ceil_div(g.N, tile) * ceil_div(g.M, tile) * g.splits);
    // one 256 x 256 tile's stages fill a CU's LDS, two of the others fit
    const unsigned most = tile == 256 ? 256 : 512, grid = End::kImage ? (unsigned)g.items : std::min((unsigned)g.items, most);
    constexpr int NA = End::kImage ? 3 : 2;
    g.round = tile == 64 ? 4 : NA == 3 ? 1 : 2;
    if constexpr (sizeof(E) == 4) {
        launch_kernel((gemm_kernel<E, End, 64, 2, 2, 4, 4, AX, BX>), dim3(grid), dim3(256), s, g, end);
    } else {
        if (tile == 256)
            launch_kernel((gemm_kernel<E, End, 256, 2, 4, 2, NA, AX, BX>), dim3(grid), dim3(512), s, g, end);
        else if (tile == 128)
            launch_kernel((gemm_kernel<E, End, 128, 2, 2, 2, NA, AX, BX>), dim3(grid), dim3(256), s, g, end);
        else
            launch_kernel((gemm_kernel<E, End, 64, 2, 2, 4, 4, AX, BX>), dim3(grid), dim3(256), s, g, end);
    }
}

template <typename T, typename Out, int PARTS>
void make_parts(const void *x, int64_t rows, int32_t d, const LossArgs *a, Out *out, Token *token, hipStream_t s) {
    const int64_t n = sizeof(Out) == 2 ? round64(rows) * (round64(d) / 8) : rows * (d / 8);
    launch_kernel((parts_kernel<T, Out, PARTS>), dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20)), dim3(256), s,
                  static_cast<const T *>(x), rows, d, a ? a->targets : static_cast<const int32_t *>(nullptr),
                  a ? a->vocab : 0, out, a ? static_cast<const float *>(a->lse) : static_cast<const float *>(nullptr),
                  a ? a->dloss : static_cast<const float *>(nullptr), a ? a->dloss_scale * a->scale : 0.f, token);
}

// A copy in blocks of rows of h or W: a bf16 plan's as they are, an fp32 plan's in
// three parts.
void make_blocks(const LossArgs &a, const void *x, int64_t rows, const LossArgs *mask, uint16_t *out, Token *token,
                 hipStream_t s) {
    if (a.bf16)
        make_parts<uint16_t, uint16_t, 1>(x, rows, a.d, mask, out, token, s);
    else
        make_parts<float, uint16_t, 3>(x, rows, a.d, mask, out, token, s);
}

// Products of parts: all pairs whose weight is 2^-16 and more, the lightest first,
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

// At most n parts of K, of whole rounds of stages (an item's last ones are zeros
// past K, not the next part's).
void split_steps(GemmArgs &g, int64_t steps, int64_t n) {
    const int64_t per = ceil_div(ceil_div(steps, n), 4) * 4;
    g.split_steps = (int32_t)per;
    g.splits = (int32_t)ceil_div(steps, per);
}

// Parts of K for a product of few tiles: as many as fill the chip's slots (one
// 256 x 256 tile a CU, two of the others) evenly, of at least eight stages.
template <class E>
void split_k(GemmArgs &g, int tile, int64_t most) {
    const int64_t tiles = ceil_div(g.M, tile) * ceil_div(g.N, tile), steps = ceil_div(g.K, step_of<E>());
    const int64_t slots = tile == 256 ? 256 : 512;
    most = std::min<int64_t>({most, steps / 8, tiles >= 8 * slots ? 1 : 8 * slots / tiles});
    int64_t best = 1;
    double best_cost = 1e30;
    for (int64_t s = 1; s <= most; ++s) {
        // rounds of the chip times a tile's stages, and a dozen stages' worth for its start and end
        const double cost = (double)ceil_div(tiles * s, slots) * ((double)ceil_div(steps, s) + 12.);
        if (cost < best_cost * 0.97) {
            best_cost = cost;
            best = s;
        }
    }
    split_steps(g, steps, best);
}

constexpr int64_t kPieceBytes = (int64_t)1 << 30;     // of P, and of W's parts, at a time
constexpr int64_t kSumBytes = (int64_t)512 << 20;     // of dh's sums in several splits
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

// dW's sums in several splits: at most 64 MB.
int64_t weight_sum_bytes(int64_t vocab, int32_t d) { return std::min<int64_t>((int64_t)64 << 20, kMostSplits * vocab * d * 4); }

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

// Whether an fp32 plan's products run on the fp32 matrix instructions, a sixteenth
// of the bf16 ones' rate, or in six products of bf16 parts: those need W's parts
// made first.
bool direct32(const LossArgs &a) { return a.n_tok <= 128; }

// Whether a bf16 plan's h (forward) and W are copied into blocks first.  Rows of
// d = 2560 put a stage's 256 lines on four of an L2's sixteen channels; in blocks
// the logits of 8192 tokens and 64,640 columns take 2.03 ms (h) and 1.92 ms (h and W)
// against 2.13 ms, their gradient's product with W 2.08 ms against 2.35 ms.  The
// copy of W costs 4 bytes a value, 0.14 ms there, so it takes this many tokens.
bool blocks_h(const LossArgs &a) { return a.bf16 && a.n_tok >= 1024 && a.vocab >= 16384; }
bool blocks_w(const LossArgs &a, bool forward) { return a.bf16 && a.n_tok >= (forward ? 12288 : 4096); }

// Parts of P, and bytes of P for a token and column.
int p_parts(const LossArgs &a) { return a.bf16 && a.dw_bf16 ? 1 : 3; }
int64_t p_bytes(const LossArgs &a) { return !a.bf16 && direct32(a) ? 4 : 2 * p_parts(a); }

}  // namespace

// The parts of a token's sums: columns of a wave by the tile's size.  One of the
// largest batch serves the smaller ones (each term grows with the batch, and the
// tiles of 64 and 128 are only taken up to some number of them).
LossLayout loss_layout(const LossArgs &a) {
    LossLayout L{};
    const int64_t v = padded(a.vocab), T = a.n_tok;
    const int64_t n128 = v / 128, n64 = v / 64, n32 = v / 32;
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = off;
        off = round256(off + bytes);
        return (size_t)o;
    };
    L.xt = take(T * 4);
    L.part = take(8 * std::max({T * n128, std::min<int64_t>(T, 128) * n32, std::min<int64_t>(T * n32, 512 * 128 * 4),
                                std::min<int64_t>(T, 128) * n64, std::min<int64_t>(T * n64, 192 * 1024 * 4)}));
    const int64_t each = a.bf16 ? 2 : 6;
    if (a.bf16 ? blocks_h(a) : !direct32(a)) L.h = take(each * round64(T) * round64(a.d));
    if (a.bf16 ? blocks_w(a, true) : !direct32(a)) L.w = take(piece_bytes(a.vocab, round64(a.d) * each));
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
    L.xt = take(a.n_tok * (int64_t)sizeof(Token));
    L.h = take((a.bf16 ? 2 : direct32(a) ? 4 : 6) * round64(a.n_tok) * round64(a.d));
    L.part = take(piece_bytes(a.vocab, p_bytes(a) * round64(a.n_tok)));
    L.sum = take(sum_bytes(a.n_tok, a.d));
    L.wsum = take(weight_sum_bytes(a.vocab, a.d));
    if (a.bf16 ? blocks_w(a, false) : !direct32(a)) L.w = take(piece_bytes(a.vocab, round64(a.d) * (a.bf16 ? 2 : 6)));
    L.total = (size_t)off;
    return L;
}

bool loss_fits(int64_t n_tok, int32_t vocab, int32_t d) {
    // items of one launch, and 31-bit offsets in a tile's rows of d or of a piece
    // of the vocabulary
    return ceil_div(n_tok, 256) * ceil_div(vocab, 256) < ((int64_t)1 << 22) &&
           ceil_div(n_tok, 256) * ceil_div(d, 256) < ((int64_t)1 << 18) && d <= (1 << 20) && vocab <= (1 << 22) &&
           n_tok <= (1 << 27);
}

namespace {

template <class E>
void forward(const LossArgs &a, hipStream_t s) {
    constexpr bool F32 = sizeof(E) == 4;
    const LossLayout L = loss_layout(a);
    char *ws = static_cast<char *>(a.ws);
    LseEnd end{a.scale, a.targets, reinterpret_cast<float *>(ws + L.xt), reinterpret_cast<float2 *>(ws + L.part), 0};
    GemmArgs g{};
    const int64_t d = a.d, V = a.vocab, T = a.n_tok;
    const bool parts = !F32 && !a.bf16;
    g.M = T;
    g.K = d;
    whole<E>(g);
    const bool bh = parts || blocks_h(a), bw = parts || blocks_w(a, true);
    const int64_t piece = bw ? piece_for(V, round64(d) * (parts ? 6 : 2)) : padded(V);
    const int tile = F32 ? 64 : tile_for(T, std::min(piece, V));
    uint16_t *h = reinterpret_cast<uint16_t *>(ws + L.h), *w = reinterpret_cast<uint16_t *>(ws + L.w);
    if (bh) make_blocks(a, a.h, T, nullptr, h, nullptr, s);
    g.a = bh ? blocks_of(h, T, d) : rows_of(a.h, T, d);
    parts_of(g, parts ? 3 : 1, parts ? 3 : 1);
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        g.N = std::min(piece, V - v0);
        end.v0 = v0;
        const char *rows = static_cast<const char *>(a.w) + v0 * d * (a.bf16 ? 2 : 4);
        if (bw) make_blocks(a, rows, g.N, nullptr, w, nullptr, s);
        g.b = bw ? blocks_of(w, g.N, d) : rows_of(rows, g.N, d);
        gemm<E, false, false>(g, end, tile, s);
    }
    launch_kernel(lse_join_kernel, dim3((unsigned)ceil_div(T, 8)), dim3(256), s, end.part, 2 * ceil_div(V, tile), T,
                  a.targets, a.vocab, end.xt, a.loss, a.lse);
}

template <class E>
void backward(const LossArgs &a, hipStream_t s) {
    constexpr bool F32 = sizeof(E) == 4;
    const LossLayout L = loss_bwd_layout(a);
    char *ws = static_cast<char *>(a.ws);
    const int64_t d = a.d, V = a.vocab, T = a.n_tok;
    const bool parts = !F32 && !a.bf16;
    const int hp = parts ? 3 : 1, pp = F32 ? 1 : p_parts(a);
    Token *token = reinterpret_cast<Token *>(ws + L.xt);
    void *h = ws + L.h, *p = ws + L.part;
    uint16_t *wp = reinterpret_cast<uint16_t *>(ws + L.w);
    float *sum = reinterpret_cast<float *>(ws + L.sum), *wsum = reinterpret_cast<float *>(ws + L.wsum);
    const bool bw = parts || blocks_w(a, false);
    if constexpr (F32)
        make_parts<float, float, 1>(a.h, T, a.d, &a, static_cast<float *>(h), token, s);
    else
        make_blocks(a, a.h, T, &a, static_cast<uint16_t *>(h), token, s);
    const Operand oh = F32 ? rows_of(h, T, d) : blocks_of(h, T, d);
    int64_t piece = piece_for(V, p_bytes(a) * round64(T));
    if (bw) piece = std::min(piece, piece_for(V, round64(d) * (parts ? 6 : 2)));
    int32_t dh_splits = 1;
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        const int64_t n = std::min(piece, V - v0), ld = round64(n);
        const Operand op = F32 ? rows_of(p, T, ld) : blocks_of(p, T, n);
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
            whole<E>(g);
            parts_of(g, hp, hp);
            const GradEnd end{a.scale, token, p, op.row64, op.part, ld, pp, v0};
            gemm<E, false, false>(g, end, F32 ? 64 : tile_for(T, n), s);
        }
        if (a.dh) {
            g.M = T;
            g.N = d;
            g.K = n;
            g.a = op;
            g.b = ow;
            parts_of(g, hp, hp);
            const int64_t steps = ceil_div(n, step_of<E>());
            const int tile = F32 ? 64 : tile_for(T, d, ceil_div(std::min(piece, V), step_of<E>()));
            // (the same split for every piece: its sums go on from one to the next)
            if (v0 == 0) {
                split_k<E>(g, tile, std::min(kMostSplits, sum_bytes(T, a.d) / (T * d * 4)));
                dh_splits = g.splits;
            } else {
                split_steps(g, steps, dh_splits);
            }
            const SumEnd end{sum, d, T * d, false, v0 > 0};
            gemm<E, false, true>(g, end, tile, s);
        }
        if (a.dw) {
            g.M = n;
            g.N = d;
            g.K = T;
            g.a = op;
            g.b = oh;
            parts_of(g, pp, hp);
            const int tile = F32 ? 64 : tile_for(n, d, ceil_div(T, step_of<E>()));
            split_k<E>(g, tile, std::min(kMostSplits, weight_sum_bytes(a.vocab, a.d) / (n * d * 4)));
            char *out = static_cast<char *>(a.dw) + v0 * d * (a.dw_bf16 ? 2 : 4);
            const bool split = g.splits > 1;
            const SumEnd end{split ? static_cast<void *>(wsum) : out, d, n * d, !split && a.dw_bf16, !split && a.accumulate};
            gemm<E, true, true>(g, end, tile, s);
            if (split) {
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

}  // namespace

void launch_loss(const LossArgs &a, hipStream_t s) {
    if (!a.bf16 && direct32(a))
        forward<float>(a, s);
    else
        forward<uint16_t>(a, s);
}

void launch_loss_bwd(const LossArgs &a, hipStream_t s) {
    if (!a.bf16 && direct32(a))
        backward<float>(a, s);
    else
        backward<uint16_t>(a, s);
}

}  // namespace engram
