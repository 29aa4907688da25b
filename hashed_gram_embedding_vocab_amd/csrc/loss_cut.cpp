// loss_cut.cpp -- sizes of the output head's cross entropy: its workspaces' regions
// and what one launch holds.
#include "loss_cut.h"

namespace engram {

// One of the largest batch serves the smaller ones: each term grows with the batch.
LossLayout loss_layout(const LossArgs &a) {
    LossLayout L{};
    const int64_t T = a.n_tok;
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = off;
        off = round256(off + bytes);
        return (size_t)o;
    };
    L.xt = take(T * 4);
    L.part = take(8 * lse_pairs(a));
    L.few = take(few_bytes(a));
    const int64_t each = a.bf16 ? 2 : 4;
    if (a.bf16 ? blocks_h(a) : !direct32(a, true)) {
        L.h = take(each * round64(T) * round64(a.d));
        L.unit = take(4 * (round64(T) + padded(a.vocab)));
    }
    if (a.bf16 ? blocks_w(a, true) : !direct32(a, true)) L.w = take(piece_bytes(a.vocab, round64(a.d) * each));
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
    const bool direct = !a.bf16 && direct32(a, false);
    L.xt = take(a.n_tok * (int64_t)sizeof(Token));
    // (a few tokens' rows stand several times: no fewer for more tokens)
    const int64_t few = a.bf16 ? p_rows(a, std::min(a.n_tok, kStack), true) : 0, rows = std::max(few, round64(a.n_tok));
    L.h = take((a.bf16 ? 2 : direct ? 4 : 6) * rows * round64(a.d));
    L.part = take(piece_bytes(a.vocab, std::max(p_bytes(a), 2 * few)));
    L.sum = take(sum_bytes(std::max(a.n_tok, a.bf16 ? 2 * std::min(a.n_tok, kStack) : 0), a.d));
    L.wsum = take(weight_sum_bytes(a.vocab, a.d));
    L.few = take(few_bytes(a));
    if (a.bf16 ? blocks_w(a, false) : !direct) L.w = take(piece_bytes(a.vocab, round64(a.d) * (a.bf16 ? 2 : 6)));
    L.total = (size_t)off;
    return L;
}

bool loss_fits(int64_t n_tok, int32_t vocab, int32_t d) {
    // items of one launch (fewer than 2^32 threads), and 31-bit offsets in a tile's
    // rows of d or of a piece of the vocabulary
    const int64_t t = ceil_div(n_tok, 256), v = ceil_div(vocab, 256), c = ceil_div(d, 256);
    return t * v < ((int64_t)1 << 22) && v * c < ((int64_t)1 << 22) && t * c < ((int64_t)1 << 18) && d <= (1 << 20) &&
           vocab <= (1 << 22) && n_tok <= (1 << 26);
}

}  // namespace engram
