// How the library cuts the output head's logits, and the workspace regions that it
// lays out for them, from its own host code.  Reads lines "dtype n_tok vocab d" (dtype
// 0: fp32, 1: bf16) and answers each with what loss_cut.h chooses and writes:
//   tile  splits  cost  pieces  bytes of the tiles' maxima and sums  bytes of their region  bytes of the workspace
//   and of the gradients' products P, dh, dW as whole rows of the vocabulary: the cost of each
#include <cstdio>

#include "loss_cut.h"

using namespace engram;

int main() {
    int bf16;
    long long n, vocab, d;
    while (std::scanf("%d %lld %lld %lld", &bf16, &n, &vocab, &d) == 4) {
        if (!loss_fits(n, (int32_t)vocab, (int32_t)d)) {
            std::puts("refused");
            continue;
        }
        LossArgs a{};
        a.n_tok = n;
        a.vocab = (int32_t)vocab;
        a.d = (int32_t)d;
        a.bf16 = bf16 != 0;
        const ForwardCut f = a.bf16              ? forward_cut<uint16_t>(a)
                             : direct32(a, true) ? forward_cut<float>(a)
                                                 : forward_cut<_Float16>(a);
        const LossLayout L = loss_layout(a);
        // (an end of the region: the next one's start, whichever that is)
        size_t end = L.total;
        for (size_t o : {L.xt, L.few, L.h, L.unit, L.w})
            if (o > L.part) end = std::min(end, o);
        const long long pairs = f.cut.splits > 1 ? 0 : 2 * ceil_div(vocab, f.cut.tile) * n;
        std::printf("%d %lld %.6g %lld %lld %zu %zu", f.cut.tile, (long long)f.cut.splits, f.cut.cost,
                    (long long)ceil_div(vocab, f.piece), 8 * pairs, end - L.part, L.total);
        auto costs = [&](auto e) {
            using E = decltype(e);
            std::printf(" %.6g %.6g %.6g\n", cut_for<E>(n, vocab, d, 1, 1, 4).cost,
                        cut_for<E>(n, d, vocab, 1, kMostSplits, 4).cost, cut_for<E>(vocab, d, n, 1, 1, 4).cost);
        };
        if (!a.bf16 && direct32(a, false))
            costs(0.f);
        else
            costs((uint16_t)0);
    }
    return 0;
}
