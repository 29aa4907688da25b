// api_operators.cpp -- host side of the operators beside the layer
// (include/engram.h): the token embedding and its gradient, layer norm and its
// gradients, the block-scaled 8-bit product and its quantisation.  Argument
// checks, workspace layout and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_internal.h"

using namespace engram;
using namespace engram::host;

namespace {

struct EmbedLayout {
    size_t order, sid, start, lead, tail, total;
};

engram_status embed_layout_of(const engram_plan_s &p, int64_t n_tok, EmbedLayout &L) {
    if (n_tok <= 0) return ENGRAM_E_INVALID_ARG;
    const int32_t d = p.cfg.d_model, V = p.cfg.vocab;
    if (n_tok > (int64_t)INT32_MAX || n_tok > kMaxElems / d || V > kMaxElems / d || !embed_bwd_fits(n_tok, V, d))
        return ENGRAM_E_UNSUPPORTED;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = round_up(off + bytes, 256);
        return o;
    };
    const size_t parts = (size_t)embed_chunks(n_tok, d) * (size_t)d * 4;
    L.order = take((size_t)n_tok * 4);
    L.sid = take((size_t)n_tok * 4);
    L.start = take(((size_t)V + 1) * 4);
    L.lead = take(parts);
    L.tail = take(parts);
    L.total = off;
    return ENGRAM_OK;
}

size_t norm_bwd_bytes(const engram_plan_s &p, int64_t n_rows) {
    return round_up((size_t)norm_bwd_blocks(n_rows, p.cfg.d_model) * 2 * (size_t)p.cfg.d_model * 4, 256);
}

// Sizes of a layer norm call.
engram_status check_norm_sizes(const engram_plan_s &p, int64_t n_rows) {
    if (n_rows <= 0) return ENGRAM_E_INVALID_ARG;
    if (!norm_fits(p.cfg.d_model) || n_rows > kMaxElems / p.cfg.d_model) return ENGRAM_E_UNSUPPORTED;
    return ENGRAM_OK;
}

size_t scale_bytes(int64_t rows, int64_t cols, int32_t block_rows) {
    return (size_t)((rows + block_rows - 1) / block_rows) * (size_t)(((cols + 127) / 128 + 3) / 4 * 4);
}

engram_status check_product_sizes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return ENGRAM_E_INVALID_ARG;
    if (K % 16 != 0 || K >= ((int64_t)1 << 22) || M > kMaxElems / K || N > kMaxElems / K || M > kMaxElems / N ||
        !product_fits(M, N, K))
        return ENGRAM_E_UNSUPPORTED;
    return ENGRAM_OK;
}

}  // namespace

extern "C" {

engram_status engram_embed(engram_plan p, const int32_t *d_tokens, int64_t n_tok, const void *d_table, float scale,
                           void *d_h, uint32_t *d_bad_tokens, hipStream_t stream) {
    if (!p || !d_tokens || !d_table || !d_h || n_tok <= 0) return ENGRAM_E_INVALID_ARG;
    if (n_tok > (int64_t)INT32_MAX || n_tok > kMaxElems / p->cfg.d_model || p->cfg.vocab > kMaxElems / p->cfg.d_model)
        return ENGRAM_E_UNSUPPORTED;
    if (!aligned16(d_tokens) || !aligned16(d_table) || !aligned16(d_h) || !std::isfinite(scale))
        return ENGRAM_E_INVALID_ARG;
    const size_t row = (size_t)p->cfg.d_model * p->elem;
    const size_t h_bytes = (size_t)p->cfg.n_branches * (size_t)n_tok * row;
    const size_t t_bytes = (size_t)p->cfg.vocab * row, tok_bytes = (size_t)n_tok * 4;
    if (overlap(d_h, h_bytes, d_table, t_bytes) || overlap(d_h, h_bytes, d_tokens, tok_bytes) ||
        overlap(d_bad_tokens, 4, d_h, h_bytes) || overlap(d_bad_tokens, 4, d_table, t_bytes) ||
        overlap(d_bad_tokens, 4, d_tokens, tok_bytes) || (reinterpret_cast<uintptr_t>(d_bad_tokens) & 3u) != 0)
        return ENGRAM_E_INVALID_ARG;
    {
        Launch l(*p, ENGRAM_K_GATHER, stream);
        launch_embed(p->cfg.dtype, d_tokens, n_tok, p->cfg.vocab, d_table, p->cfg.d_model, p->cfg.n_branches, scale,
                     d_h, d_bad_tokens, stream);
    }
    return last_launch_status();
}

size_t engram_embed_backward_workspace_size(engram_plan p, int64_t n_tok) {
    EmbedLayout L, S;
    if (!p || embed_layout_of(*p, n_tok, L) != ENGRAM_OK) return 0;
    // either kind of chunk takes more for more tokens, but a long batch's are
    // four times the length: the batch before them can take more than this one
    const int64_t n_short = embed_short_tokens(p->cfg.d_model);
    if (n_short < n_tok && embed_layout_of(*p, n_short, S) == ENGRAM_OK) return std::max(L.total, S.total);
    return L.total;
}

engram_status engram_embed_backward(engram_plan p, const int32_t *d_tokens, int64_t n_tok, const void *d_dh,
                                    float scale, uint32_t flags, float *d_dtable, void *d_workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
    if (!p || !d_tokens || !d_dh || !d_dtable || !d_workspace) return ENGRAM_E_INVALID_ARG;
    if (flags & ~(uint32_t)ENGRAM_GRAD_ACCUMULATE) return ENGRAM_E_INVALID_ARG;
    EmbedLayout L;
    const engram_status st = embed_layout_of(*p, n_tok, L);
    if (st != ENGRAM_OK) return st;
    if (workspace_bytes < L.total || !aligned256(d_workspace)) return ENGRAM_E_INVALID_ARG;
    if (!aligned16(d_tokens) || !aligned16(d_dh) || !aligned16(d_dtable) || !std::isfinite(scale))
        return ENGRAM_E_INVALID_ARG;
    const size_t d = (size_t)p->cfg.d_model;
    const size_t dh_bytes = (size_t)p->cfg.n_branches * (size_t)n_tok * d * p->elem;
    const size_t dt_bytes = (size_t)p->cfg.vocab * d * 4, tok_bytes = (size_t)n_tok * 4;
    if (overlap(d_dtable, dt_bytes, d_dh, dh_bytes) || overlap(d_dtable, dt_bytes, d_tokens, tok_bytes) ||
        overlap(d_workspace, L.total, d_dh, dh_bytes) || overlap(d_workspace, L.total, d_dtable, dt_bytes) ||
        overlap(d_workspace, L.total, d_tokens, tok_bytes))
        return ENGRAM_E_INVALID_ARG;
    char *base = static_cast<char *>(d_workspace);
    EmbedBwdArgs a{};
    a.tokens = d_tokens;
    a.dh = d_dh;
    a.dtable = d_dtable;
    a.order = reinterpret_cast<uint32_t *>(base + L.order);
    a.sid = reinterpret_cast<int32_t *>(base + L.sid);
    a.start = reinterpret_cast<uint32_t *>(base + L.start);
    a.lead = reinterpret_cast<float *>(base + L.lead);
    a.tail = reinterpret_cast<float *>(base + L.tail);
    a.n_tok = n_tok;
    a.vocab = p->cfg.vocab;
    a.d = p->cfg.d_model;
    a.n_branches = p->cfg.n_branches;
    a.scale = scale;
    a.accumulate = (flags & ENGRAM_GRAD_ACCUMULATE) != 0;
    {
        Launch l(*p, ENGRAM_K_BWD_TABLE, stream);
        launch_embed_bwd(p->cfg.dtype, a, stream);
    }
    return last_launch_status();
}

engram_status engram_layer_norm(engram_plan p, const void *d_x, int64_t n_rows, const float *d_gamma,
                                const float *d_beta, float eps, void *d_y, float *d_mean, float *d_rstd,
                                hipStream_t stream) {
    if (!p || !d_x || !d_gamma || !d_y || !(eps >= 0.f) || !std::isfinite(eps)) return ENGRAM_E_INVALID_ARG;
    const engram_status st = check_norm_sizes(*p, n_rows);
    if (st != ENGRAM_OK) return st;
    if (!aligned16(d_x) || !aligned16(d_gamma) || !aligned16(d_y) || (d_beta && !aligned16(d_beta)) ||
        (d_mean && !aligned16(d_mean)) || (d_rstd && !aligned16(d_rstd)))
        return ENGRAM_E_INVALID_ARG;
    const size_t bytes = (size_t)n_rows * p->cfg.d_model * p->elem, col = (size_t)p->cfg.d_model * 4;
    const size_t rows = (size_t)n_rows * 4;
    if ((d_y != d_x && overlap(d_y, bytes, d_x, bytes)) || overlap(d_y, bytes, d_gamma, col) ||
        overlap(d_y, bytes, d_beta, col) || overlap(d_mean, rows, d_x, bytes) || overlap(d_rstd, rows, d_x, bytes) ||
        overlap(d_mean, rows, d_y, bytes) || overlap(d_rstd, rows, d_y, bytes) || overlap(d_mean, rows, d_rstd, rows) ||
        overlap(d_mean, rows, d_gamma, col) || overlap(d_mean, rows, d_beta, col) ||
        overlap(d_rstd, rows, d_gamma, col) || overlap(d_rstd, rows, d_beta, col))
        return ENGRAM_E_INVALID_ARG;
    NormArgs a{};
    a.x = d_x;
    a.y = d_y;
    a.gamma = d_gamma;
    a.beta = d_beta;
    a.mean = d_mean;
    a.rstd = d_rstd;
    a.n_rows = n_rows;
    a.d = p->cfg.d_model;
    a.eps = eps;
    {
        Launch l(*p, ENGRAM_K_AUX, stream);
        launch_norm(p->cfg.dtype, a, stream);
    }
    return last_launch_status();
}

size_t engram_layer_norm_backward_workspace_size(engram_plan p, int64_t n_rows) {
    if (!p || check_norm_sizes(*p, n_rows) != ENGRAM_OK) return 0;
    return norm_bwd_bytes(*p, n_rows);
}

engram_status engram_layer_norm_backward(engram_plan p, const void *d_x, const void *d_dy, int64_t n_rows,
                                         const float *d_gamma, const float *d_mean, const float *d_rstd,
                                         uint32_t flags, void *d_dx, float *d_dgamma, float *d_dbeta,
                                         void *d_workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!p || !d_x || !d_dy || !d_gamma || !d_mean || !d_rstd || !d_dx || !d_dgamma || !d_workspace)
        return ENGRAM_E_INVALID_ARG;
    if (flags & ~(uint32_t)ENGRAM_GRAD_ACCUMULATE) return ENGRAM_E_INVALID_ARG;
    const engram_status st = check_norm_sizes(*p, n_rows);
    if (st != ENGRAM_OK) return st;
    const size_t ws = norm_bwd_bytes(*p, n_rows);
    if (workspace_bytes < ws || !aligned256(d_workspace)) return ENGRAM_E_INVALID_ARG;
    if (!aligned16(d_x) || !aligned16(d_dy) || !aligned16(d_gamma) || !aligned16(d_mean) || !aligned16(d_rstd) ||
        !aligned16(d_dx) || !aligned16(d_dgamma) || (d_dbeta && !aligned16(d_dbeta)))
        return ENGRAM_E_INVALID_ARG;
    const size_t bytes = (size_t)n_rows * p->cfg.d_model * p->elem, col = (size_t)p->cfg.d_model * 4;
    const size_t rows = (size_t)n_rows * 4;
    // what is written: dx (in place of x or dy if the caller likes), dgamma, dbeta, the workspace
    const void *outs[4] = {d_dx, d_dgamma, d_dbeta, d_workspace};
    const size_t out_n[4] = {bytes, col, col, ws};
    const void *ins[5] = {d_x, d_dy, d_gamma, d_mean, d_rstd};
    const size_t in_n[5] = {bytes, bytes, col, rows, rows};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (!(i == 0 && j < 2 && outs[0] == ins[j]) && overlap(outs[i], out_n[i], ins[j], in_n[j]))
                return ENGRAM_E_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], out_n[i], outs[j], out_n[j])) return ENGRAM_E_INVALID_ARG;
    }
    NormArgs a{};
    a.x = d_x;
    a.dy = d_dy;
    a.dx = d_dx;
    a.gamma = d_gamma;
    a.mean = const_cast<float *>(d_mean);
    a.rstd = const_cast<float *>(d_rstd);
    a.part = static_cast<float *>(d_workspace);
    a.dgamma = d_dgamma;
    a.dbeta = d_dbeta;
    a.n_rows = n_rows;
    a.d = p->cfg.d_model;
    a.accumulate = (flags & ENGRAM_GRAD_ACCUMULATE) != 0;
    {
        Launch l(*p, ENGRAM_K_BWD_FUSE, stream);
        launch_norm_bwd(p->cfg.dtype, a, stream);
    }
    return last_launch_status();
}

engram_status engram_quantize_fp8(engram_plan p, const void *d_x, int64_t rows, int64_t cols, int32_t block_rows,
                                  uint32_t flags, void *d_q, uint8_t *d_scales, hipStream_t stream) {
    if (!p || !d_x || !d_q || !d_scales || rows <= 0 || cols <= 0) return ENGRAM_E_INVALID_ARG;
    if (block_rows != 1 && block_rows != 128) return ENGRAM_E_INVALID_ARG;
    if (flags & ~(uint32_t)ENGRAM_QUANTIZE_TRANSPOSE) return ENGRAM_E_INVALID_ARG;
    if (rows > kMaxElems / cols || rows > (int64_t)INT32_MAX || cols > (int64_t)INT32_MAX) return ENGRAM_E_UNSUPPORTED;
    if (!aligned16(d_x) || !aligned16(d_q) || !aligned16(d_scales)) return ENGRAM_E_INVALID_ARG;
    QuantArgs a{};
    a.x = d_x;
    a.q = d_q;
    a.scales = d_scales;
    a.rows = rows;
    a.cols = cols;
    a.block_rows = block_rows;
    a.transpose = (flags & ENGRAM_QUANTIZE_TRANSPOSE) != 0;
    const size_t n = (size_t)rows * (size_t)cols;
    const size_t sb = a.transpose ? scale_bytes(cols, rows, block_rows) : scale_bytes(rows, cols, block_rows);
    if (overlap(d_q, n, d_x, n * p->elem) || overlap(d_scales, sb, d_x, n * p->elem) || overlap(d_scales, sb, d_q, n))
        return ENGRAM_E_INVALID_ARG;
    {
        Launch l(*p, ENGRAM_K_AUX, stream);
        launch_quantize(p->cfg.dtype, a, stream);
    }
    return last_launch_status();
}

size_t engram_matmul_fp8_workspace_size(engram_plan p, int64_t M, int64_t N, int64_t K) {
    if (!p || check_product_sizes(M, N, K) != ENGRAM_OK) return 0;
    return product_workspace_most(M, N, K);
}

engram_status engram_matmul_fp8(engram_plan p, const void *d_a, const uint8_t *d_a_scales, int32_t a_block_rows,
                                const void *d_b, const uint8_t *d_b_scales, int32_t b_block_rows, int64_t M, int64_t N,
                                int64_t K, void *d_c, engram_dtype c_dtype, void *d_workspace, size_t workspace_bytes,
                                hipStream_t stream) {
    if (!p || !d_a || !d_a_scales || !d_b || !d_b_scales || !d_c) return ENGRAM_E_INVALID_ARG;
    if ((a_block_rows != 1 && a_block_rows != 128) || (b_block_rows != 1 && b_block_rows != 128))
        return ENGRAM_E_INVALID_ARG;
    if (c_dtype != ENGRAM_F32 && c_dtype != ENGRAM_BF16) return ENGRAM_E_INVALID_ARG;
    const engram_status st = check_product_sizes(M, N, K);
    if (st != ENGRAM_OK) return st;
    if (!aligned16(d_a) || !aligned16(d_a_scales) || !aligned16(d_b) || !aligned16(d_b_scales) || !aligned16(d_c))
        return ENGRAM_E_INVALID_ARG;
    const size_t ws = product_workspace(M, N, K);
    if (ws > 0 && (!d_workspace || workspace_bytes < ws || !aligned256(d_workspace))) return ENGRAM_E_INVALID_ARG;
    const size_t c_bytes = (size_t)M * (size_t)N * (c_dtype == ENGRAM_BF16 ? 2 : 4);
    const void *ins[4] = {d_a, d_b, d_a_scales, d_b_scales};
    const size_t in_n[4] = {(size_t)M * (size_t)K, (size_t)N * (size_t)K, scale_bytes(M, K, a_block_rows),
                            scale_bytes(N, K, b_block_rows)};
    for (int i = 0; i < 4; ++i)
        if (overlap(d_c, c_bytes, ins[i], in_n[i]) || (ws > 0 && overlap(d_workspace, ws, ins[i], in_n[i])))
            return ENGRAM_E_INVALID_ARG;
    if (ws > 0 && overlap(d_workspace, ws, d_c, c_bytes)) return ENGRAM_E_INVALID_ARG;
    ProductArgs a{};
    a.a = static_cast<const uint8_t *>(d_a);
    a.b = static_cast<const uint8_t *>(d_b);
    a.a_scales = d_a_scales;
    a.b_scales = d_b_scales;
    a.c = d_c;
    a.ws = d_workspace;
    a.M = M;
    a.N = N;
    a.K = K;
    a.a_block_rows = a_block_rows;
    a.b_block_rows = b_block_rows;
    a.out_bf16 = c_dtype == ENGRAM_BF16;
    {
        Launch l(*p, ENGRAM_K_GEMM, stream);
        launch_product(a, stream);
    }
    return last_launch_status();
}

}  // extern "C"
