// loss_cut.h -- the host side of the output head's cross entropy (loss.hip) as far
// as it is arithmetic on sizes: how a product is cut into tiles and parts of K, how the
// vocabulary is cut into pieces, and which regions a workspace has.
#pragma once

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "engram_internal.h"

namespace engram {

constexpr int kBlock = 64;  // rows and columns of a block of the workspaces' matrices

// What the gradient of a token's logits needs: lse, the factor g_t scale (0 for a
// token that does not count) and the target.
struct Token {
    float lse, factor;
    int32_t target, unused;
};

inline int64_t round64(int64_t x) { return (x + kBlock - 1) / kBlock * kBlock; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class E>
constexpr int64_t step_of() {
    return 128 / (int64_t)sizeof(E);
}

// How a product is cut: square tiles, and parts of K.  The tile and the parts are
// those that should take least, by what a stage takes on a CU (measured, us): 1.48
// with one workgroup of 256 x 256, 0.92 with two of 128 x 128 (0.62 with one),
// 0.44 with two of 64 x 64 (0.30), and at its start and end a few us more, which
// grow with the bytes of a result.  (A 256 x 256 tile's 1.33 PFLOP/s are 1.05 of
// 128 x 128 and 0.53 of 64 x 64; but 96 tiles of 64 x 64 are six of 256 x 256.)
// fp32 tiles are 64 x 64 (0.95, 0.55) or 32 x 32 (0.58, 0.36): 33 tokens x 1000 x 256
// are 16 of the one or 64 of the other, 13.4 us against 10.0.  Parts of K cost a
// second launch that joins them.  Against the best of each tile forced, and of
// parts or none, the choice lost less than 5% in 92 shapes but two (5 and 7%).
struct Cut {
    int tile;
    int64_t splits;
    double cost;
};

// A type's largest tile may come in any number, and so may 64 x 64 over 64 rows and less;
// of the others a launch may have so many (lse_pairs counts on that).
template <class E>
constexpr int largest_tile() {
    return sizeof(E) == 4 ? 64 : std::is_same<E, _Float16>::value ? 128 : 256;
}
constexpr int64_t most_items(int tile) { return tile == 128 ? 2048 : tile == 64 ? 1024 : 512; }

template <class E>
bool may_tile(int tile, int64_t M, int64_t N) {
    return tile == largest_tile<E>() || (tile == 64 && M <= 64) || ceil_div(M, tile) * ceil_div(N, tile) <= most_items(tile);
}

template <class E>
Cut cut_for(int64_t M, int64_t N, int64_t K, int segs, int64_t most, int out_bytes, bool walks = false) {
    struct Rate {
        int tile;
        double one, two, start1, start2, byte1, byte2;
    };
    constexpr bool F32 = sizeof(E) == 4, PARTS = std::is_same<E, _Float16>::value;
    static constexpr Rate kRates16[3] = {{64, 0.30, 0.44, 3., 4., 0.25, 0.5},
                                         {128, 0.62, 0.92, 5., 6., 0.7, 1.3},
                                         {256, 1.48, 1.48, 5., 5., 2.3, 2.3}};
    // (a stage of fp32: 32 k at a sixteenth of the rate)
    static constexpr Rate kRates32[2] = {{32, 0.36, 0.58, 3., 4., 0.1, 0.2}, {64, 0.55, 0.95, 4., 5., 0.25, 0.5}};
    // (fp16: three products a stage of 32 k)
    static constexpr Rate kRatesParts[2] = {{64, 0.35, 0.55, 3., 4., 0.25, 0.5}, {128, 0.75, 1.20, 5., 6., 0.7, 1.3}};
    auto &rates = [&]() -> auto & {
        if constexpr (F32) return kRates32;
        else if constexpr (PARTS) return kRatesParts;
        else return kRates16;
    }();
    Cut best{0, 1, 1e30};  // (there is a better one: of the largest tile)
    const int64_t steps = ceil_div(K, step_of<E>());
    for (const Rate &r : rates) {
        if (walks ? r.tile == 256 || r.tile == 32 : !may_tile<E>(r.tile, M, N)) continue;
        const int64_t tiles = ceil_div(M, r.tile) * ceil_div(N, r.tile), slots = r.tile == 256 ? 256 : 512;
        for (int64_t n = 1; n == 1 || (n <= most && n * 4 <= steps); n = n < 16 ? n + 1 : n + n / 4) {
            const int64_t items = tiles * n, full = items / slots, rest = items % slots;
            const double each = (double)((walks ? ceil_div(steps, 2) * 2 : ceil_div(steps, n)) * segs);
            const int bytes = n > 1 ? 4 : out_bytes;
            const double less = walks ? 0.6 : 1.;  // (the next item's first stages land while one ends)
            double t = (double)full * (each * r.two + less * (r.start2 + r.byte2 * bytes));
            if (rest > 0)
                t += rest <= 256 ? each * r.one + less * (r.start1 + r.byte1 * bytes) : each * r.two + less * (r.start2 + r.byte2 * bytes);
            if (n > 1) t += 4. + (double)(n * M) * (double)N * 4. / 4.5e6;
            if (t < best.cost * 0.98) best = Cut{r.tile, n, t};
        }
    }
    return best;
}

constexpr int64_t kPieceBytes = (int64_t)1 << 30;     // of P, and of W's parts, at a time
constexpr int64_t kSumBytes = (int64_t)512 << 20;     // of dh's sums in several splits
constexpr int64_t kMostSplits = 64;
constexpr int64_t kFewBytes = (int64_t)32 << 20;      // of a few tokens' logits in several splits

inline int64_t padded(int64_t vocab) { return ceil_div(vocab, 256) * 256; }

// Columns of the vocabulary taken at a time: `bytes` for each of them may come
// to kPieceBytes, but at least 256 columns.
inline int64_t piece_for(int64_t vocab, int64_t bytes) {
    const int64_t most = std::max<int64_t>(256, kPieceBytes / bytes / 256 * 256);
    const int64_t n = ceil_div(padded(vocab), most);
    return ceil_div(ceil_div(padded(vocab), n), 256) * 256;
}
// What such a piece takes at most; it never falls as `bytes` grows.
inline int64_t piece_bytes(int64_t vocab, int64_t bytes) {
    return std::max(256 * bytes, std::min(kPieceBytes, padded(vocab) * bytes));
}

// (`rows`: twice the tokens where P has two parts below each other)
inline int64_t sum_bytes(int64_t rows, int32_t d) {
    const int64_t one = rows * d * 4;
    return std::max(one, std::min(kSumBytes, kMostSplits * one));
}

// dW's sums in several splits: at most 64 MB.
inline int64_t weight_sum_bytes(int64_t vocab, int32_t d) { return std::min<int64_t>((int64_t)64 << 20, kMostSplits * vocab * d * 4); }

inline int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

// The tokens up to which an fp32 plan's products run on the fp32 matrix instructions, a sixteenth
// of the bf16 ones' rate, or as products of parts (three of fp16 parts forward, six of
// bf16 parts backward), which need W's parts made first: as long as a second
// reading of W takes (some 100 tokens' products), and where V is small their
// launches (a time of its own) and, forward, tiles of too few workgroups along
// all of d.  Measured, us, instructions of fp32 against parts: forward 59 tokens x
// 61016 x 2832 233 : 484, 517 x 32000 x 1024 377 : 162, 521 x 773 x 5952 72 : 82,
// 1000 x 773 x 5952 136 : 86, 1000 x 1000 x 256 14 : 16, 6000 x 1000 x 256 46 : 30; backward
// 59 x 61016 x 2832 857 : 1374, 275 x 22940 x 1496 702 : 567, 521 x 773 x 5952
// 207 : 174, 1000 x 1000 x 256 46 : 59.  In 49 shapes the rule lost up to 8%, and 19% of two
// short ones whose second row of tiles was nearly empty (80 x 8962 x 1216, 57 : 47).
inline int64_t direct_tokens(const LossArgs &a, bool forward) {
    return forward ? 80 + (300000000 / a.d + 350000) / a.vocab : 100 + 800000000 / a.d / a.vocab;
}
inline bool direct32(const LossArgs &a, bool forward) { return a.n_tok <= direct_tokens(a, forward); }

// Whether a bf16 plan's h (forward) and W are copied into blocks first: where their rows
// are no whole lines of 128 bytes, so that each piece of 128 bytes touches two.  Measured,
// us, rows as they are : copied (whole calls, the copies' 4 bytes a value among them):
// h   1024 tokens x 116,816 x 2568 668 : 628, 8192 x 232,912 x 1288 4832 : 4552,
//     2048 x 24,312 x 2056 181 : 179; 8192 x 3648 x 4104 215 : 229
// W   forward 16,384 x 38,936 x 2568 2956 : 2607, 12,288 x 15,520 x 1288 461 : 445; 8192 x
//     24,312 x 2056 682 : 672, 4096 x 12,176 x 4104 329 : 352.  Backward 4096 x 155,272 x
//     1288 5015 : 4825, 4096 x 30,000 x 1000 723 : 668; 2560 x 97,272 x 2056 2903 : 2903,
//     1536 x 48,728 x 4104 1715 : 1756
// Of whole lines the copies cost: forward 0 to 3% in 11 shapes of 8192 tokens and more,
// backward 0 to 3% in 22 widths of 256 to 8192 (6144 x 106,528 x 2816 9022 : 9143, 8192 x
// 64,000 x 4096 9477 : 9565), and saved 1 to 3% at d = 2560 and 5120 (8192 x 129,280 x 2560
// 13,081 : 12,678; dh over 160 million weights reads 9.6 GB : 4.6 past the L2s).  No rule was
// found that names these two: 1280, 7680, 10,240 and 12,800, 2496 and 2624 lose or are even.
inline bool split_lines(const LossArgs &a) { return a.bf16 && a.d % 64 != 0; }
inline bool blocks_h(const LossArgs &a) { return split_lines(a) && a.n_tok >= 1024 && a.vocab >= 16384; }
inline bool blocks_w(const LossArgs &a, bool forward) { return split_lines(a) && a.n_tok >= (forward ? 12288 : 4096); }

// A bf16 plan's few tokens: the parts of P are further rows of it, and h's rows
// stand as often, so that W is still read once for dh, where its bytes are what
// counts, with two parts of P (for dW two, or three for an fp32 one).  A few tokens'
// gradients are a few products, whose one rounding to bf16 would not average out
// (up to 2^-8 of their norm, twice what a result's own rounding is): 33 tokens x 1000
// x 256 are 1.7e-3 of dh's norm from 64 bits instead of 2.7e-3 (22 -> 26 us), 33 x 129280
// x 2560 take 705 us instead of 775 (fp32 dW; bf16 541 and 546).  128 tokens would take a fifth longer,
// and their roundings average out (2.4e-3, where very many end too).
constexpr int64_t kStack = 64;
inline bool stacked(const LossArgs &a) { return a.bf16 && a.n_tok <= kStack; }

// Parts of P, rows of it and of the copy of h, and bytes of P for a column.
inline int p_parts(const LossArgs &a, bool stack) { return !a.bf16 || !a.dw_bf16 ? 3 : stack ? 2 : 1; }
inline int64_t p_rows(const LossArgs &a, int64_t n_tok, bool stack) { return round64(stack ? p_parts(a, true) * n_tok : n_tok); }
inline int64_t p_bytes(const LossArgs &a) {
    const int64_t each = !a.bf16 && direct32(a, false) ? 4 : stacked(a) ? 2 : 2 * p_parts(a, false);
    return each * p_rows(a, a.n_tok, stacked(a));
}

inline int64_t round8(int64_t x) { return (x + 7) / 8 * 8; }
inline int64_t few_bytes(const LossArgs &a) { return std::min(kFewBytes, kMostSplits * a.n_tok * round8(a.vocab) * 4); }

constexpr int kFewThreads = 1024, kFewEach = 8;  // of a workgroup for each of a few tokens
// A few tokens of a small vocabulary: the logits in parts of K, where that is
// faster than whole rows by the tiles there are (122 tokens x 75 x 7680 in fp32: two
// workgroups would do 240 stages each).  splits 1: not.
template <class E>
Cut few_cut(const LossArgs &a, int64_t N, int64_t K, int segs, int out_bytes) {
    const Cut whole = cut_for<E>(a.n_tok, N, K, segs, 1, out_bytes);
    const int64_t one = a.n_tok * round8(a.vocab) * 4;
    if (one > kFewBytes / 2 || (out_bytes == 0 && N > kFewThreads * kFewEach)) return whole;
    const Cut parts = cut_for<E>(a.n_tok, N, K, segs, few_bytes(a) / one, 4);
    // (the forward's maxima and sums are joined by a launch of their own anyway, which
    // takes less than one of a workgroup for each token)
    const double more = out_bytes ? 1. : (double)a.n_tok / 100 - 3.;
    return parts.splits > 1 && parts.cost + more < whole.cost ? parts : whole;
}

// How the forward runs: whether h and W are copied into blocks first, columns of the
// vocabulary at a time, and the cut of their logits.
struct ForwardCut {
    bool blocks_h, blocks_w;
    int64_t piece;
    Cut cut;
};
// (W's copy has two fp16 parts in an fp32 plan)
inline int64_t forward_piece(const LossArgs &a, bool copied) {
    return copied ? piece_for(a.vocab, round64(a.d) * (a.bf16 ? 2 : 4)) : padded(a.vocab);
}
template <class E>
ForwardCut forward_cut(const LossArgs &a) {
    constexpr bool F32 = sizeof(E) == 4, F16 = std::is_same<E, _Float16>::value;
    ForwardCut f;
    f.blocks_h = F16 || (!F32 && blocks_h(a));
    f.blocks_w = F16 || (!F32 && blocks_w(a, true));
    f.piece = forward_piece(a, f.blocks_w);
    const int64_t n = std::min<int64_t>(f.piece, a.vocab), k = F16 ? (a.d + 31) / 32 * 64 : a.d;
    f.cut = F16 ? cut_for<E>(a.n_tok, n, k, 1, 1, 0) : few_cut<E>(a, n, k, 1, 0);
    return f;
}

// Pairs of a maximum and a sum that the forward's tiles may write: two of each row of a
// tile, over the whole vocabulary, of whatever tiles may_tile() allows a launch, which
// makes one piece of it.  It never falls as tokens are added.
inline int64_t lse_pairs(const LossArgs &a) {
    const bool copied = a.bf16 ? blocks_w(a, true) : !direct32(a, true);
    const int64_t T = a.n_tok, V = a.vocab, pieces = ceil_div(V, forward_piece(a, copied));
    auto all = [&](int tile, int64_t rows) { return 2 * ceil_div(V, tile) * rows; };
    auto few = [&](int tile) { return std::min(all(tile, T), pieces * most_items(tile) * 2 * tile); };
    const int64_t small = std::max({all(64, std::min<int64_t>(T, 64)), few(64), few(32)});
    if (a.bf16) return std::max({small, few(128), all(256, T)});
    return std::max({small, all(128, T), all(64, std::min(T, direct_tokens(a, true)))});
}

}  // namespace engram
