// api_ends.cpp -- host side of the operators at a model's ends
// (include/engram.h): RMS norm with the residual's addition and its gradients,
// the output head's cross entropy and its gradients, the clipping of gradients.
// Argument checks, workspace layout and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "host_internal.h"

using namespace engram;
using namespace engram::host;

namespace {

// A buffer of a call.
struct Buf {
    const void *p;
    size_t n;
};
bool overlap(const Buf &a, const Buf &b) { return engram::host::overlap(a.p, a.n, b.p, b.n); }
bool aligned16_or_null(const void *p) { return !p || aligned16(p); }

// Sizes of an RMS norm call.
engram_status check_rms_sizes(const engram_plan_s &p, int64_t n_rows) {
    if (n_rows <= 0) return ENGRAM_E_INVALID_ARG;
    if (!norm_fits(p.cfg.d_model) || n_rows > kMaxElems / p.cfg.d_model) return ENGRAM_E_UNSUPPORTED;
    return ENGRAM_OK;
}

size_t rms_bwd_bytes(const engram_plan_s &p, int64_t n_rows) {
    return round_up((size_t)rms_bwd_blocks(n_rows, p.cfg.d_model) * (size_t)p.cfg.d_model * 4, 256);
}

// (the logits are taken as powers of two: scale / ln 2 has to be finite too)
bool scale_fits(float scale) { return std::fabs(scale) <= 0x1p127f; }

engram_status check_loss_sizes(const engram_plan_s &p, int64_t n_tok) {
    if (n_tok <= 0) return ENGRAM_E_INVALID_ARG;
    if (!loss_fits(n_tok, p.cfg.vocab, p.cfg.d_model)) return ENGRAM_E_UNSUPPORTED;
    return ENGRAM_OK;
}

LossArgs loss_args(const engram_plan_s &p, int64_t n_tok) {
    LossArgs a{};
    a.n_tok = n_tok;
    a.vocab = p.cfg.vocab;
    a.d = p.cfg.d_model;
    a.bf16 = p.cfg.dtype == ENGRAM_BF16;
    a.scale = a.dloss_scale = 1.f;
    return a;
}

// Whether dweight_dtype is one the plan's gradients can have.
engram_status check_dweight(const engram_plan_s &p, engram_dtype dt) {
    if (dt != ENGRAM_F32 && dt != ENGRAM_BF16) return ENGRAM_E_INVALID_ARG;
    return dt == ENGRAM_BF16 && p.cfg.dtype != ENGRAM_BF16 ? ENGRAM_E_UNSUPPORTED : ENGRAM_OK;
}

}  // namespace

extern "C" {

engram_status engram_rms_norm(engram_plan p, const void *d_x, const void *d_residual, int64_t n_rows,
                              const float *d_gamma, float eps, void *d_total, void *d_y, void *d_q, uint8_t *d_scales,
                              float *d_rrms, hipStream_t stream) {
    if (!p || !d_x || !d_gamma || !(eps >= 0.f) || !std::isfinite(eps)) return ENGRAM_E_INVALID_ARG;
    if (!d_residual != !d_total || !d_q != !d_scales || (!d_y && !d_q)) return ENGRAM_E_INVALID_ARG;
    const engram_status st = check_rms_sizes(*p, n_rows);
    if (st != ENGRAM_OK) return st;
    if (!aligned16(d_x) || !aligned16(d_gamma) || !aligned16_or_null(d_residual) || !aligned16_or_null(d_total) ||
        !aligned16_or_null(d_y) || !aligned16_or_null(d_q) || !aligned16_or_null(d_scales) || !aligned16_or_null(d_rrms))
        return ENGRAM_E_INVALID_ARG;
    const size_t n = (size_t)n_rows * p->cfg.d_model, bytes = n * p->elem;
    const Buf ins[3] = {{d_x, bytes}, {d_residual, bytes}, {d_gamma, (size_t)p->cfg.d_model * 4}};
    const Buf outs[5] = {{d_total, bytes},
                         {d_y, bytes},
                         {d_q, n},
                         {d_scales, (size_t)n_rows * (size_t)((p->cfg.d_model + 511) / 512 * 4)},
                         {d_rrms, (size_t)n_rows * 4}};
    for (int i = 0; i < 5; ++i) {
        // (total and y may each take the place of x or of the residual: rows are read before they are written)
        for (int j = 0; j < 3; ++j)
            if (!(i < 2 && j < 2 && outs[i].p == ins[j].p) && overlap(outs[i], ins[j])) return ENGRAM_E_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return ENGRAM_E_INVALID_ARG;
    }
    if (d_residual && d_residual != d_x && overlap(ins[0], ins[1]) && (d_total == d_x || d_total == d_residual ||
        d_y == d_x || d_y == d_residual))
        return ENGRAM_E_INVALID_ARG;  // in place of one of two inputs that lie across each other
    RmsArgs a{};
    a.x = d_x;
    a.res = d_residual;
    a.total = d_total;
    a.y = d_y;
    a.q = static_cast<uint8_t *>(d_q);
    a.scales = d_scales;
    a.gamma = d_gamma;
    a.rrms = d_rrms;
    a.n_rows = n_rows;
    a.d = p->cfg.d_model;
    a.eps = eps;
    {
        Launch l(*p, ENGRAM_K_AUX, stream);
        launch_rms(p->cfg.dtype, a, stream);
    }
    return last_launch_status();
}

size_t engram_rms_norm_backward_workspace_size(engram_plan p, int64_t n_rows) {
    if (!p || check_rms_sizes(*p, n_rows) != ENGRAM_OK) return 0;
    return rms_bwd_bytes(*p, n_rows);
}

engram_status engram_rms_norm_backward(engram_plan p, const void *d_s, const void *d_dy, const void *d_dtotal,
                                       int64_t n_rows, const float *d_gamma, const float *d_rrms, uint32_t flags,
                                       void *d_dx, float *d_dgamma, void *d_workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
    if (!p || !d_s || !d_dy || !d_gamma || !d_rrms || !d_dx || !d_dgamma || !d_workspace) return ENGRAM_E_INVALID_ARG;
    if (flags & ~(uint32_t)ENGRAM_GRAD_ACCUMULATE) return ENGRAM_E_INVALID_ARG;
    const engram_status st = check_rms_sizes(*p, n_rows);
    if (st != ENGRAM_OK) return st;
    const size_t ws = rms_bwd_bytes(*p, n_rows);
    if (workspace_bytes < ws || !aligned256(d_workspace)) return ENGRAM_E_INVALID_ARG;
    if (!aligned16(d_s) || !aligned16(d_dy) || !aligned16_or_null(d_dtotal) || !aligned16(d_gamma) ||
        !aligned16(d_rrms) || !aligned16(d_dx) || !aligned16(d_dgamma))
        return ENGRAM_E_INVALID_ARG;
    const size_t bytes = (size_t)n_rows * p->cfg.d_model * p->elem, col = (size_t)p->cfg.d_model * 4;
    const Buf ins[5] = {{d_s, bytes}, {d_dy, bytes}, {d_dtotal, bytes}, {d_gamma, col}, {d_rrms, (size_t)n_rows * 4}};
    const Buf outs[3] = {{d_dx, bytes}, {d_dgamma, col}, {d_workspace, ws}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (!(i == 0 && j < 3 && outs[0].p == ins[j].p) && overlap(outs[i], ins[j])) return ENGRAM_E_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return ENGRAM_E_INVALID_ARG;
    }
    RmsArgs a{};
    a.x = d_s;
    a.dy = d_dy;
    a.ds = d_dtotal;
    a.dx = d_dx;
    a.gamma = d_gamma;
    a.rrms = const_cast<float *>(d_rrms);
    a.part = static_cast<float *>(d_workspace);
    a.dgamma = d_dgamma;
    a.n_rows = n_rows;
    a.d = p->cfg.d_model;
    a.accumulate = (flags & ENGRAM_GRAD_ACCUMULATE) != 0;
    {
        Launch l(*p, ENGRAM_K_BWD_FUSE, stream);
        launch_rms_bwd(p->cfg.dtype, a, stream);
    }
    return last_launch_status();
}

size_t engram_cross_entropy_workspace_size(engram_plan p, int64_t n_tok) {
    if (!p || check_loss_sizes(*p, n_tok) != ENGRAM_OK) return 0;
    return loss_layout(loss_args(*p, n_tok)).total;
}

engram_status engram_cross_entropy(engram_plan p, const void *d_h, const void *d_weight, const int32_t *d_targets,
                                   int64_t n_tok, float scale, float *d_loss, float *d_lse, void *d_workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    if (!p || !d_h || !d_weight || !d_targets || !d_loss || !d_lse || !d_workspace || !scale_fits(scale))
        return ENGRAM_E_INVALID_ARG;
    const engram_status st = check_loss_sizes(*p, n_tok);
    if (st != ENGRAM_OK) return st;
    LossArgs a = loss_args(*p, n_tok);
    const size_t ws = loss_layout(a).total;
    if (workspace_bytes < ws || !aligned256(d_workspace)) return ENGRAM_E_INVALID_ARG;
    if (!aligned16(d_h) || !aligned16(d_weight) || !aligned16(d_targets) || !aligned16(d_loss) || !aligned16(d_lse))
        return ENGRAM_E_INVALID_ARG;
    const size_t row = (size_t)p->cfg.d_model * p->elem, tok = (size_t)n_tok * 4;
    const Buf ins[3] = {{d_h, (size_t)n_tok * row}, {d_weight, (size_t)p->cfg.vocab * row}, {d_targets, tok}};
    const Buf outs[3] = {{d_loss, tok}, {d_lse, tok}, {d_workspace, ws}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlap(outs[i], ins[j])) return ENGRAM_E_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return ENGRAM_E_INVALID_ARG;
    }
    a.h = d_h;
    a.w = d_weight;
    a.targets = d_targets;
    a.loss = d_loss;
    a.lse = d_lse;
    a.ws = d_workspace;
    a.scale = scale;
    {
        Launch l(*p, ENGRAM_K_GEMM, stream);
        launch_loss(a, stream);
    }
    return last_launch_status();
}

size_t engram_cross_entropy_backward_workspace_size(engram_plan p, int64_t n_tok, engram_dtype dweight_dtype) {
    if (!p || check_loss_sizes(*p, n_tok) != ENGRAM_OK || check_dweight(*p, dweight_dtype) != ENGRAM_OK) return 0;
    LossArgs a = loss_args(*p, n_tok);
    a.dw_bf16 = dweight_dtype == ENGRAM_BF16;
    return loss_bwd_layout(a).total;
}

engram_status engram_cross_entropy_backward(engram_plan p, const void *d_h, const void *d_weight,
                                            const int32_t *d_targets, int64_t n_tok, float scale, const float *d_lse,
                                            const float *d_dloss, float dloss_scale, uint32_t flags, void *d_dh,
                                            void *d_dweight, engram_dtype dweight_dtype, void *d_workspace,
                                            size_t workspace_bytes, hipStream_t stream) {
    if (!p || !d_h || !d_weight || !d_targets || !d_lse || (!d_dh && !d_dweight) || !d_workspace)
        return ENGRAM_E_INVALID_ARG;
    if (!scale_fits(scale) || !std::isfinite(dloss_scale) || (flags & ~(uint32_t)ENGRAM_GRAD_ACCUMULATE))
        return ENGRAM_E_INVALID_ARG;
    engram_status st = check_loss_sizes(*p, n_tok);
    if (st == ENGRAM_OK) st = check_dweight(*p, dweight_dtype);
    if (st != ENGRAM_OK) return st;
    LossArgs a = loss_args(*p, n_tok);
    a.dw_bf16 = dweight_dtype == ENGRAM_BF16;
    const size_t ws = loss_bwd_layout(a).total;
    if (workspace_bytes < ws || !aligned256(d_workspace)) return ENGRAM_E_INVALID_ARG;
    if (!aligned16(d_h) || !aligned16(d_weight) || !aligned16(d_targets) || !aligned16(d_lse) ||
        !aligned16_or_null(d_dloss) || !aligned16_or_null(d_dh) || !aligned16_or_null(d_dweight))
        return ENGRAM_E_INVALID_ARG;
    const size_t row = (size_t)p->cfg.d_model * p->elem, tok = (size_t)n_tok * 4;
    const Buf ins[5] = {{d_h, (size_t)n_tok * row}, {d_weight, (size_t)p->cfg.vocab * row}, {d_targets, tok}, {d_lse, tok},
                        {d_dloss, tok}};
    const Buf outs[3] = {{d_dh, (size_t)n_tok * row},
                         {d_dweight, (size_t)p->cfg.vocab * (size_t)p->cfg.d_model * (a.dw_bf16 ? 2 : 4)},
                         {d_workspace, ws}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (overlap(outs[i], ins[j])) return ENGRAM_E_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return ENGRAM_E_INVALID_ARG;
    }
    a.h = d_h;
    a.w = d_weight;
    a.targets = d_targets;
    a.lse = const_cast<float *>(d_lse);
    a.dloss = d_dloss;
    a.dh = d_dh;
    a.dw = d_dweight;
    a.ws = d_workspace;
    a.scale = scale;
    a.dloss_scale = dloss_scale;
    a.accumulate = (flags & ENGRAM_GRAD_ACCUMULATE) != 0;
    {
        Launch l(*p, ENGRAM_K_BWD_GEMM, stream);
        launch_loss_bwd(a, stream);
    }
    return last_launch_status();
}

size_t engram_clip_grads_workspace_size(engram_plan p, int32_t n_grads) {
    return p && n_grads > 0 ? clip_workspace(n_grads) : 0;
}

engram_status engram_clip_grads(engram_plan p, const engram_grad *grads, int32_t n_grads, float max_norm, float *d_norm,
                                void *d_workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!p || !grads || n_grads <= 0 || !d_norm || !d_workspace || !(max_norm > 0.f)) return ENGRAM_E_INVALID_ARG;
    const size_t ws = clip_workspace(n_grads);
    if (workspace_bytes < ws || !aligned256(d_workspace) || !aligned16(d_norm)) return ENGRAM_E_INVALID_ARG;
    try {
        struct Span {
            uintptr_t from, to;
            bool alone;  // no other buffer may share a byte with it
        };
        std::vector<Span> spans;
        spans.reserve((size_t)n_grads * 3 + 2);
        auto add = [&](const void *q, size_t n, bool alone) {
            if (q && n) spans.push_back(Span{reinterpret_cast<uintptr_t>(q), reinterpret_cast<uintptr_t>(q) + n, alone});
        };
        int64_t total = 0;
        for (int32_t i = 0; i < n_grads; ++i) {
            const engram_grad &g = grads[i];
            if (g.dtype != ENGRAM_F32 && g.dtype != ENGRAM_BF16) return ENGRAM_E_INVALID_ARG;
            if (g.n_groups < 0 || g.rows < 0 || g.row_len < 0) return ENGRAM_E_INVALID_ARG;
            if (g.n_groups == 0 || g.rows == 0 || g.row_len == 0) continue;
            if (g.rows > kMaxElems / g.row_len || g.n_groups > kMaxElems / (g.rows * g.row_len)) return ENGRAM_E_UNSUPPORTED;
            const int64_t n = g.n_groups * g.rows * g.row_len;
            // (a group takes whole pieces: many short groups are more of them than their values say)
            if ((total += std::max(n, clip_chunks(g) * 4096)) > kMaxElems) return ENGRAM_E_UNSUPPORTED;
            if (!g.data || !aligned16(g.data) || !aligned16_or_null(g.out) ||
                (reinterpret_cast<uintptr_t>(g.row_counts) & 3u) != 0)
                return ENGRAM_E_INVALID_ARG;
            const size_t bytes = (size_t)n * (g.dtype == ENGRAM_BF16 ? 2 : 4);
            add(g.data, bytes, true);
            if (g.out != g.data) add(g.out, bytes, true);
            add(g.row_counts, (size_t)g.n_groups * 4, false);
        }
        add(d_norm, 8, true);
        add(d_workspace, ws, true);
        // (only counts may be shared: a gradient listed twice would count twice)
        std::sort(spans.begin(), spans.end(), [](const Span &a, const Span &b) { return a.from < b.from; });
        uintptr_t end = 0, end_alone = 0;
        for (const Span &s : spans) {
            if (s.from < end_alone || (s.alone && s.from < end)) return ENGRAM_E_INVALID_ARG;
            end = std::max(end, s.to);
            if (s.alone) end_alone = std::max(end_alone, s.to);
        }
    } catch (const std::bad_alloc &) {
        return ENGRAM_E_NOMEM;
    }
    {
        Launch l(*p, ENGRAM_K_AUX, stream);
        launch_clip(grads, n_grads, max_norm, d_norm, static_cast<double *>(d_workspace), stream);
    }
    return last_launch_status();
}

}  // extern "C"
