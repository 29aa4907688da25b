"""The operators at a model's ends on the GPU (RMS norm with the residual's
addition, cross entropy of the output head, clipping of gradients) against plain
64-bit implementations.

Tolerances count roundings: u = 2^-24 is fp32's half step.  A product over K is a
chain of ceil(K / 32) matrix instructions for each product of parts, whose
rounded adds and the sums of 32 inside one are taken as off by 2 u each of the
magnitudes' sum; an output rounded to bf16 is off by 2^-8 of its value (fp32: u).
"""

import math

import pytest
import torch

from test_gpu_operators import Guarded, close, gen, half_step, make_plan, randn, tdt, zipf_ids

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = ("bf16", "f32")


def nan_like(t):
    """A buffer whose old values would show."""
    return t.fill_(math.nan)


# ---------------------------------------------------------------- cross entropy


def head(dtype, n_tok, vocab, d, scale, seed, gpu, skip=True):
    """A head's inputs: some tokens nearly certain, a few that do not count."""
    w = randn((vocab, d), dtype, seed, 1.0 / math.sqrt(d) / abs(scale))
    y = zipf_ids(n_tok, vocab, seed + 1, bad=skip)
    h = torch.randn((n_tok, d), generator=gen(seed + 2))
    sure = torch.rand((n_tok, 1), generator=gen(seed + 3)) * 10
    h = (h + sure * scale * w[y.clamp(0, vocab - 1).long()].float()).to(tdt(dtype))
    return h.to(gpu), w.to(gpu), y.to(gpu)


def chain(k, segs):
    return 2 * (segs * -(-k // 32) + 40)


class HeadRef:
    """Losses, gradients and bounds of their errors in 64 bits, some tokens at a time."""

    def __init__(self, h, w, y, scale, dtype):
        self.h, self.w, self.y, self.scale = h.double(), w.double(), y.long(), scale
        self.V, self.d = w.shape
        self.segs = 1 if dtype == "bf16" else 6
        self.dtype = dtype
        self.counts = (self.y >= 0) & (self.y < self.V)

    def logits(self, at):
        """Logits of tokens `at` and how far the kernel's may be off: sums, and what
        products of parts leave out (5 u of three bf16 parts; 12 u of two fp16 parts,
        whose sums are chains of three products and not of six)."""
        h = self.h[at]
        x = h @ self.w.t() * self.scale
        mag = h.abs() @ self.w.abs().t() * abs(self.scale)
        return x, (chain(self.d, self.segs) + 6) * U * mag + U * x.abs()

    def forward(self):
        n = len(self.y)
        out = [torch.zeros(n, dtype=torch.float64, device=self.h.device) for _ in range(4)]
        for at in self.counts.nonzero()[:, 0].split(1024):
            x, e = self.logits(at)
            lse = x.logsumexp(1)
            xy = x.gather(1, self.y[at][:, None])[:, 0]
            # exponentials and their sum: 300 roundings at most, and those of the join
            off = e.amax(1) + 300 * U + 4 * U * (lse.abs() + x.amax(1).abs())
            out[0][at], out[1][at] = lse - xy, lse
            out[2][at], out[3][at] = 2 * off + 4 * U * xy.abs(), off
        return out

    def backward(self, lse, g, dw_dtype, p_bits=8):
        """dh, dW and their bounds, from the lse that the kernel is given.  p_bits: of a
        bf16 plan's P, for dh and a bf16 dW."""
        n, V, d = len(self.y), self.V, self.d
        dev = self.h.device
        dh, dh_off = (torch.zeros((n, d), dtype=torch.float64, device=dev) for _ in range(2))
        dw, dw_off = (torch.zeros((V, d), dtype=torch.float64, device=dev) for _ in range(2))
        rh = 2.0 ** -p_bits if self.dtype == "bf16" else 2.0 ** -22  # what P's parts leave out, and the products of parts
        rw = 2.0 ** -22 if self.dtype == "f32" else 2.0 ** -p_bits if dw_dtype == torch.bfloat16 else 2.0 ** -16
        sh, sw = chain(V, self.segs) + 40, chain(n, 6 if self.dtype == "f32" else 2) + 40
        for at in self.counts.nonzero()[:, 0].split(1024):
            x, e = self.logits(at)
            l = lse[at].double()[:, None]
            f = (g[at].double() * self.scale)[:, None]
            p = (x - l).exp()
            off = p * (e + 4 * U * (x - l).abs() + U * l.abs() + 8 * U)
            p[torch.arange(len(at), device=dev), self.y[at]] -= 1.0
            p, off = p * f, (off + 2 * U * p.abs()) * f.abs() + 2.0 ** -126
            h, w = self.h[at], self.w
            mag_h, mag_w = p.abs() @ w.abs(), p.abs().t() @ h.abs()
            dh[at] = p @ w
            dh_off[at] = off @ w.abs() + (rh + sh * U) * mag_h
            dw += p.t() @ h
            dw_off += off.t() @ h.abs() + (rw + sw * U) * mag_w
        return dh, dh_off + half_step(self.dtype) * dh.abs(), dw, dw_off + torch.finfo(dw_dtype).eps / 2 * dw.abs()


HEADS = [  # n_tok, vocab, d, scale
    (1, 1, 8, 1.0), (1, 50, 64, 1.0), (2, 300, 72, -0.5), (63, 257, 264, 1.0), (64, 4099, 128, 0.25),
    (65, 1000, 256, 1.0), (130, 33, 520, 1.0), (333, 1000, 256, 0.0625), (300, 5003, 72, 1.0), (1100, 2111, 136, 1.0),
    (513, 260, 8, 1.0), (2049, 50, 64, 1.0), (700, 16500, 64, 2.0), (3, 70000, 128, 1.0),
    # h in blocks, W in blocks (backward; forward), long rows of few tokens, many tiles of 128
    (1030, 16500, 72, 1.0), (4100, 300, 136, 1.0), (12290, 270, 72, 1.0), (5, 130, 5000, 1.0), (70, 90, 4104, -0.3),
    (150, 1100, 3080, 1.0), (260, 9000, 200, 1.0), (1500, 1500, 264, 1.0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok,vocab,d,scale", HEADS)
def test_cross_entropy(gpu, dtype, n_tok, vocab, d, scale):
    p = make_plan(dtype, d, vocab)
    h, w, y = head(dtype, n_tok, vocab, d, scale, 3, gpu)
    loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok), scale=scale)
    ref, ref_lse, off, off_lse = (t.cpu() for t in HeadRef(h, w, y, scale, dtype).forward())
    close(loss, ref, off, "loss")
    close(lse, ref_lse, off_lse, "lse")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok,vocab,d,scale", [(1, 242, 208, 0.5), (40, 300, 64, 1.0), (9, 5000, 136, -1.0), (300, 1, 64, 1.0),
                                                 (700, 5003, 264, 1.0), (2500, 1000, 512, -0.5), (70, 90, 4104, 1.0)])
def test_certain_tokens_keep_their_digits(gpu, dtype, n_tok, vocab, d, scale):
    """A loss is log(1 + exp(a)) with a = log sum of the others' exponentials over the
    target's: its derivative 1 - exp(-loss) is small where the loss is, and so is what
    an error of the logits makes of it, down to losses far below lse's own rounding."""
    p = make_plan(dtype, d, vocab)
    w = randn((vocab, d), dtype, 3, 1.0 / math.sqrt(d) / abs(scale))
    y = (torch.arange(n_tok) * 5 % vocab).to(torch.int32)
    # logits of about 0 to 35 at the target
    h = torch.randn((n_tok, d), generator=gen(4)) + torch.linspace(0, 35, n_tok).flip(0)[:, None] * scale * w[y.long()].float()
    h, w, y = h.to(tdt(dtype)).to(gpu), w.to(gpu), y.to(gpu)
    loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok), scale=scale)
    r = HeadRef(h, w, y, scale, dtype)
    _, ref_lse, off, off_lse = (t.cpu() for t in r.forward())
    x = r.logits(torch.arange(n_tok, device=gpu))[0]
    own = x.gather(1, y.long()[:, None])
    rest = x.scatter(1, y.long()[:, None], -math.inf).logsumexp(1)
    ref = torch.log1p((rest - own[:, 0]).exp()).cpu()
    close(loss, ref, 1.01 * (1 - (-ref).exp()) * off + 8 * U * ref, "loss")
    close(lse, ref_lse, off_lse, "lse")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok,vocab,d", [(1, 50, 64), (70, 257, 72), (700, 5003, 264), (1100, 17000, 72)])
def test_logits_scaled_to_nothing(gpu, dtype, n_tok, vocab, d):
    """scale 0: all logits are 0, loss and lse log(vocab), no gradient."""
    p = make_plan(dtype, d, vocab)
    h, w, y = head(dtype, n_tok, vocab, d, 1.0, 3, gpu)
    loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok), scale=0.0)
    ref = torch.where((y >= 0) & (y < vocab), math.log(vocab), 0.0).double().cpu()
    close(loss, ref, 300 * U + 4 * U * ref, "loss")
    close(lse, ref, 300 * U + 4 * U * ref, "lse")
    dh, dw = nan_like(torch.empty_like(h)), nan_like(torch.empty_like(w))
    p.engram_cross_entropy_backward(h, w, y, lse, None, dh, dw, p.cross_entropy_backward_workspace(n_tok, w.dtype), scale=0.0)
    assert not dh.count_nonzero() and not dw.count_nonzero()


GRADS = [("bf16", torch.bfloat16), ("bf16", torch.float32), ("f32", torch.float32)]


def check_backward(gpu, dtype, dw_dtype, n_tok, vocab, d, scale, with_dloss=True):
    p = make_plan(dtype, d, vocab)
    h, w, y = head(dtype, n_tok, vocab, d, scale, 5, gpu)
    ref = HeadRef(h, w, y, scale, dtype)
    lse = ref.forward()[1].float()
    dloss = torch.rand(n_tok, generator=gen(8)).to(gpu) if with_dloss else None
    dh = nan_like(torch.empty_like(h))
    dw = nan_like(torch.empty((vocab, d), dtype=dw_dtype, device=gpu))
    ws = p.cross_entropy_backward_workspace(n_tok, dw_dtype)
    ws.fill_(255)  # NaN in every type
    p.engram_cross_entropy_backward(h, w, y, lse, dloss, dh, dw, ws, scale=scale, dloss_scale=0.125)
    g = (dloss.double() if with_dloss else torch.ones(n_tok, device=gpu, dtype=torch.float64)) * 0.125
    rdh, off_h, rdw, off_w = (t.cpu() for t in ref.backward(lse, g, dw_dtype))
    close(dh, rdh, off_h, "dh")
    close(dw, rdw, off_w, "dw")
    assert not dh[~ref.counts].count_nonzero()
    return p, (h, w, y, lse, dloss), (dh, dw), ws


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
@pytest.mark.parametrize("n_tok,vocab,d,scale", HEADS)
def test_cross_entropy_backward(gpu, dtype, dw_dtype, n_tok, vocab, d, scale):
    p, (h, w, y, lse, dloss), (dh, dw), ws = check_backward(gpu, dtype, dw_dtype, n_tok, vocab, d, scale)
    # one of both alone, and again: the same bits
    dh2, dw2 = torch.empty_like(dh), torch.empty_like(dw)
    p.engram_cross_entropy_backward(h, w, y, lse, dloss, None, dw2, ws, scale=scale, dloss_scale=0.125)
    p.engram_cross_entropy_backward(h, w, y, lse, dloss, dh2, None, ws, scale=scale, dloss_scale=0.125)
    assert torch.equal(dw2, dw) and torch.equal(dh2, dh)
    # accumulated: once more what is there
    p.engram_cross_entropy_backward(h, w, y, lse, dloss, None, dw2, ws, scale=scale, dloss_scale=0.125, flags=8)
    assert torch.allclose(dw2.double(), 2 * dw.double(), rtol=2.0 ** -7 if dw_dtype == torch.bfloat16 else 1e-5,
                          atol=2e-5 * float(dw.double().abs().max()) if dw_dtype == torch.float32 else
                          2.0 ** -8 * float(dw.double().abs().max()))


@pytest.mark.parametrize("dw_dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("n_tok", (1, 3, 20, 21, 22, 32, 33, 43, 64, 65))
@pytest.mark.parametrize("vocab,d", [(1, 8), (77, 72), (300, 4104), (9001, 264), (40000, 64)])
def test_few_tokens_keep_two_parts_of_p(gpu, vocab, d, n_tok, dw_dtype):
    """Two roundings to bf16 in turn leave 2^-16 of P, up to 64 tokens; one alone 2^-8."""
    p = make_plan("bf16", d, vocab)
    h, w, y = head("bf16", n_tok, vocab, d, 1.0, 5, gpu)
    y[n_tok // 2] = -1  # (its h reaches nothing)
    ref = HeadRef(h, w, y, 1.0, "bf16")
    lse, g = ref.forward()[1].float(), torch.rand(n_tok, generator=gen(8)).to(gpu)
    h[n_tok // 2] = math.nan
    dh, dw = nan_like(torch.empty_like(h)), Guarded((vocab, d), dw_dtype, gpu)
    ws = Guarded((p.engram_cross_entropy_backward_workspace_size(n_tok, dw_dtype),), torch.uint8, gpu)
    p.engram_cross_entropy_backward(h, w, y, lse, g, dh, dw.t, ws.t)
    rdh, off_h, rdw, off_w = (t.cpu() for t in ref.backward(lse, g, dw_dtype, p_bits=16 if n_tok <= 64 else 8))
    close(dh, rdh, off_h, "dh")
    close(dw.t, rdw, off_w, "dw")
    once = dw.t.clone()
    p.engram_cross_entropy_backward(h, w, y, lse, g, None, dw.t, ws.t, flags=8)
    assert torch.equal(dw.t, 2 * once) or dw_dtype == torch.bfloat16
    torch.cuda.synchronize()
    assert dw.whole() and ws.whole()


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
def test_cross_entropy_backward_without_dloss(gpu, dtype, dw_dtype):
    check_backward(gpu, dtype, dw_dtype, 200, 777, 136, 1.0, with_dloss=False)


PATHS = [(9, 300, 72), (200, 1000, 264), (600, 5003, 136), (1100, 17000, 72), (4200, 270, 72)]


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
@pytest.mark.parametrize("n_tok,vocab,d", PATHS)
def test_tokens_that_do_not_count_may_hold_anything(gpu, dtype, dw_dtype, n_tok, vocab, d):
    """NaN and infinity in their h, lse and dloss reach nothing; their own results are zeros."""
    p = make_plan(dtype, d, vocab)
    h, w, y = head(dtype, n_tok, vocab, d, 1.0, 3, gpu, skip=False)
    out = torch.arange(n_tok, device=gpu) % 3 == 1
    out[-1] = True
    y[out] = torch.tensor([-1, vocab, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=gpu)[torch.arange(int(out.sum()), device=gpu) % 4]
    dloss = torch.rand(n_tok, generator=gen(8)).to(gpu)
    results = []
    for junk in (0.0, math.nan, math.inf):
        h[out] = junk
        loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
        p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
        assert not loss[out].count_nonzero() and not lse[out].count_nonzero()
        lse_in, g = lse.clone(), dloss.clone()
        lse_in[out] = g[out] = junk
        dh, dw = nan_like(torch.empty_like(h)), nan_like(torch.empty((vocab, d), dtype=dw_dtype, device=gpu))
        ws = p.cross_entropy_backward_workspace(n_tok, dw_dtype)
        ws.fill_(255)
        p.engram_cross_entropy_backward(h, w, y, lse_in, g, dh, dw, ws)
        assert not dh[out].count_nonzero() and torch.isfinite(dh).all() and torch.isfinite(dw).all()
        results.append((loss, lse, dh, dw))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
@pytest.mark.parametrize("n_tok,vocab,d", PATHS)
def test_tokens_whose_loss_has_no_gradient(gpu, dtype, dw_dtype, n_tok, vocab, d):
    """dloss 0: no part in either gradient, whatever their h and lse hold."""
    p = make_plan(dtype, d, vocab)
    h, w, y = head(dtype, n_tok, vocab, d, 1.0, 3, gpu, skip=False)
    loss, lse = torch.empty(n_tok, device=gpu), torch.empty(n_tok, device=gpu)
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
    out = torch.arange(n_tok, device=gpu) % 3 == 1
    out[-1] = True
    dloss = torch.rand(n_tok, generator=gen(8)).to(gpu) + 0.1
    dloss[out] = 0.0
    results = []
    for junk in (None, math.nan, math.inf, -math.inf):
        hj, lj = h.clone(), lse.clone()
        if junk is not None:
            hj[out], lj[out] = junk, junk
        dh, dw = nan_like(torch.empty_like(h)), nan_like(torch.empty((vocab, d), dtype=dw_dtype, device=gpu))
        ws = p.cross_entropy_backward_workspace(n_tok, dw_dtype)
        ws.fill_(255)
        p.engram_cross_entropy_backward(hj, w, y, lj, dloss, dh, dw, ws)
        assert not dh[out].count_nonzero() and dh[~out].any(1).all() and torch.isfinite(dw).all()
        results.append((dh, dw))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


@pytest.mark.parametrize("n_tok,vocab,d", [(40, 300, 520), (700, 5003, 520)])
def test_rows_of_far_apart_sizes(gpu, n_tok, vocab, d):
    """fp32 rows of 2^100 and 2^-100: their products may be where neither is."""
    p = make_plan("f32", d, vocab)
    half = d // 2
    h = torch.zeros((n_tok, d))
    h[:, :half] = randn((n_tok, half), "f32", 1) * torch.where(torch.arange(n_tok) % 2 == 0, 2.0 ** 100, 2.0 ** -100)[:, None]
    w = randn((vocab, d), "f32", 2, 2.0 ** -103)
    w[:10, :half] = 0.0  # logits 0, from rows whose units are 2^100 and 2^60
    w[:10, half:] *= 2.0 ** 100
    w[:10, half:] *= 2.0 ** 63
    y = (torch.arange(n_tok) * 7 % vocab).to(torch.int32)
    h, w, y = h.to(gpu), w.to(gpu), y.to(gpu)
    loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
    ref, ref_lse, off, off_lse = (t.cpu() for t in HeadRef(h, w, y, 1.0, "f32").forward())
    close(loss, ref, off, "loss")
    close(lse, ref_lse, off_lse, "lse")


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
def test_no_token_counts(gpu, dtype, dw_dtype):
    for n_tok, vocab, d in PATHS:
        p = make_plan(dtype, d, vocab)
        h, w, y = head(dtype, n_tok, vocab, d, 1.0, 3, gpu)
        y.fill_(-1)
        loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
        p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
        dh, dw = nan_like(torch.empty_like(h)), nan_like(torch.empty((vocab, d), dtype=dw_dtype, device=gpu))
        ws = p.cross_entropy_backward_workspace(n_tok, dw_dtype)
        p.engram_cross_entropy_backward(h, w, y, lse, None, dh, dw, ws)
        assert not any(t.count_nonzero() for t in (loss, lse, dh, dw))
        dw.fill_(3.0)
        p.engram_cross_entropy_backward(h, w, y, lse, None, dh, dw, ws, flags=8)
        assert (dw == 3.0).all()


def test_nan_stays_in_its_token(gpu):
    for n_tok, vocab, d in PATHS:
        p = make_plan("bf16", d, vocab)
        h, w, y = head("bf16", n_tok, vocab, d, 1.0, 3, gpu, skip=False)

        def call():
            loss, lse = torch.empty(n_tok, device=gpu), torch.empty(n_tok, device=gpu)
            p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
            dh, dw = torch.empty_like(h), torch.empty_like(w)
            p.engram_cross_entropy_backward(h, w, y, lse, None, dh, dw, p.cross_entropy_backward_workspace(n_tok, torch.bfloat16))
            return loss, lse, dh

        clean = call()
        h[4, 3] = math.nan
        got = call()
        ok = torch.arange(n_tok, device=gpu) != 4
        for a, b in zip(clean, got):
            assert torch.equal(a[ok], b[ok]) and b[4].isnan().all()
        h[4, 3] = 0.0
        w[vocab // 2, 1] = math.nan
        assert all(t.isnan().all() for t in call())


@pytest.mark.parametrize("dtype", DTYPES)
def test_far_logits(gpu, dtype):
    """Logits of some ten thousand, all the same, and one far above: no overflow, and
    the loss of the one that is certain is zero."""
    for n_tok, vocab, d in PATHS:
        p = make_plan(dtype, d, vocab)
        h, w = torch.ones((n_tok, d), dtype=tdt(dtype), device=gpu), torch.zeros((vocab, d), dtype=tdt(dtype), device=gpu)
        y = (torch.arange(n_tok, device=gpu) % vocab).to(torch.int32)
        loss, lse = torch.empty(n_tok, device=gpu), torch.empty(n_tok, device=gpu)
        ws = p.cross_entropy_workspace(n_tok)
        for level in (0.0, 128.0, -128.0):
            w.fill_(level)
            p.engram_cross_entropy(h, w, y, loss, lse, ws)
            want = level * d + math.log(vocab)
            assert (lse.double() - want).abs().max() <= 4 * U * abs(want) + 1e-6
            assert (loss.double() - math.log(vocab)).abs().max() <= 4 * U * abs(want) + 1e-6
        w.fill_(-128.0)
        w[vocab - 1] = 128.0
        y.fill_(vocab - 1)
        p.engram_cross_entropy(h, w, y, loss, lse, ws)
        assert (loss == 0).all() and (lse == 128.0 * d).all()
        y.fill_(0)
        p.engram_cross_entropy(h, w, y, loss, lse, ws)
        assert (loss == 256.0 * d).all()
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        p.engram_cross_entropy_backward(h, w, y, lse, None, dh, dw, p.cross_entropy_backward_workspace(n_tok, tdt(dtype)))
        assert (dh == 256.0).all() and (dw[0] == -n_tok).all() and (dw[vocab - 1] == n_tok).all() and not dw[1:-1].any()


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
def test_cross_entropy_backward_in_pieces(gpu, dtype, dw_dtype):
    """More than 1 GB of the logits' gradients: pieces of the vocabulary, dh's sums going on."""
    check_backward(gpu, dtype, dw_dtype, 8190, 70010, 72, 1.0)


def test_cross_entropy_in_pieces(gpu):
    """An fp32 plan's W in more than 1 GB of parts."""
    n_tok, vocab, d = 150, 140001, 2056
    p = make_plan("f32", d, vocab)
    h, w, y = head("f32", n_tok, vocab, d, 1.0, 3, gpu)
    loss, lse = torch.empty(n_tok, device=gpu), torch.empty(n_tok, device=gpu)
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
    ref, ref_lse, off, off_lse = (t.cpu() for t in HeadRef(h, w, y, 1.0, "f32").forward())
    close(loss, ref, off, "loss")
    close(lse, ref_lse, off_lse, "lse")


def test_cross_entropy_past_32_bits(gpu):
    """Offsets past 2^31 and 2^32 bytes in W, its gradient, h and dh: the results of
    few rows and columns there are those of a small call."""
    torch.cuda.empty_cache()
    # W: all rows but the last 300 far below, so that these alone make the loss
    vocab, d, n_tok, tail = 270000, 8200, 5, 300
    p, small = make_plan("bf16", d, vocab), make_plan("bf16", d, tail)
    h = randn((n_tok, d), "bf16", 1).abs().to(gpu)
    w = torch.full((vocab, d), -1.0, dtype=torch.bfloat16, device=gpu)  # logits of thousands below zero
    w[-tail:] = randn((tail, d), "bf16", 2, 0.01).to(gpu)
    y = torch.tensor([0, 7, 299, 100, 298], dtype=torch.int32, device=gpu)
    out = [[torch.empty(n_tok, device=gpu) for _ in range(2)] for _ in range(2)]
    p.engram_cross_entropy(h, w, y + (vocab - tail), *out[0], p.cross_entropy_workspace(n_tok))
    small.engram_cross_entropy(h, w[-tail:], y, *out[1], small.cross_entropy_workspace(n_tok))
    for a, b in zip(*out):
        assert torch.allclose(a, b, rtol=1e-6, atol=1e-6)
    dh, dw = torch.empty_like(h), nan_like(torch.empty_like(w))
    dhs, dws = torch.empty_like(h), torch.empty_like(w[-tail:])
    p.engram_cross_entropy_backward(h, w, y + (vocab - tail), out[1][1], None, dh, dw,
                                    p.cross_entropy_backward_workspace(n_tok, torch.bfloat16))
    small.engram_cross_entropy_backward(h, w[-tail:], y, out[1][1], None, dhs, dws,
                                        small.cross_entropy_backward_workspace(n_tok, torch.bfloat16))
    # (both round P of 8 bits; its sums' order differs)
    assert (dw[-tail:].double() - dws.double()).abs().max() <= 2.0 ** -7 * float(dws.double().abs().max())
    assert (dh.double() - dhs.double()).abs().max() <= 2.0 ** -7 * float(dhs.double().abs().max())
    assert not dw[:-tail].count_nonzero()
    del w, dw
    torch.cuda.empty_cache()
    n_tok, d, vocab, tail = (1 << 20) + 77, 2056, 40, 301
    p = make_plan("bf16", d, vocab)
    w = randn((vocab, d), "bf16", 3, 0.02).to(gpu)
    h = torch.zeros((n_tok, d), dtype=torch.bfloat16, device=gpu)
    h[-tail:] = randn((tail, d), "bf16", 4).to(gpu)
    y = torch.full((n_tok,), -1, dtype=torch.int32, device=gpu)
    y[-tail:] = zipf_ids(tail, vocab, 5, bad=False).to(gpu)
    loss, lse, dh = (torch.empty(n_tok, device=gpu), torch.empty(n_tok, device=gpu), nan_like(torch.empty_like(h)))
    dw = torch.empty((vocab, d), device=gpu)
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
    p.engram_cross_entropy_backward(h, w, y, lse, None, dh, dw, p.cross_entropy_backward_workspace(n_tok))
    ref = HeadRef(h[-tail:], w, y[-tail:], 1.0, "bf16")
    r = [t.cpu() for t in ref.forward()]
    close(loss[-tail:], r[0], r[2], "loss")
    g = torch.ones(tail, dtype=torch.float64, device=gpu)
    rdh, off_h, rdw, off_w = (t.cpu() for t in ref.backward(lse[-tail:], g, torch.float32))
    close(dh[-tail:], rdh, off_h, "dh")
    close(dw, rdw, off_w + 2 * (-(-n_tok // 32)) * 3 * U * rdw.abs(), "dw")  # (a longer chain, of zeros)
    assert not dh[:-tail].count_nonzero() and not loss[:-tail].count_nonzero()
    del h, dh
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
def test_cross_entropy_in_the_largest_batchs_workspace(gpu, dtype, dw_dtype):
    p = make_plan(dtype, 136, 3000)
    big = p.cross_entropy_workspace(5000), p.cross_entropy_backward_workspace(5000, dw_dtype)
    for n_tok in (1, 21, 33, 64, 65, 700, 2049):
        h, w, y = head(dtype, n_tok, 3000, 136, 1.0, 3, gpu)
        res = []
        for f, b in (big, (p.cross_entropy_workspace(n_tok), p.cross_entropy_backward_workspace(n_tok, dw_dtype))):
            f.fill_(255), b.fill_(255)
            loss, lse, dh = torch.empty(n_tok, device=gpu), torch.empty(n_tok, device=gpu), torch.empty_like(h)
            dw = torch.empty((3000, 136), dtype=dw_dtype, device=gpu)
            p.engram_cross_entropy(h, w, y, loss, lse, f)
            p.engram_cross_entropy_backward(h, w, y, lse, None, dh, dw, b)
            res.append((loss, lse, dh, dw))
        assert all(torch.equal(a, b) for a, b in zip(*res))


def test_cross_entropy_backward_is_the_difference_of_the_loss(gpu):
    """Along random directions, by central differences of the loss in 64 bits."""
    n, V, d, scale = 150, 700, 136, 0.7
    p = make_plan("f32", d, V)
    h, w, y = head("f32", n, V, d, scale, 7, gpu)
    dloss = torch.rand(n, generator=gen(9)).to(gpu)
    loss, lse = torch.empty(n, device=gpu), torch.empty(n, device=gpu)
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n), scale=scale)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    p.engram_cross_entropy_backward(h, w, y, lse, dloss, dh, dw, p.cross_entropy_backward_workspace(n), scale=scale)
    counts = (y >= 0) & (y < V)

    def total(hh, ww):
        x = hh @ ww.t() * scale
        each = x.logsumexp(1) - x.gather(1, y.clamp(0, V - 1).long()[:, None])[:, 0]
        return (each * dloss.double())[counts].sum()

    for seed in range(3):
        uh, uw = randn((n, d), "f32", 20 + seed).to(gpu).double(), randn((V, d), "f32", 30 + seed).to(gpu).double()
        for dirs, got in (((uh, 0 * uw), (dh.double() * uh).sum()), ((0 * uh, uw), (dw.double() * uw).sum())):
            step = 1e-4  # the third derivative's term: about step^2 of the difference
            diff = (total(h.double() + step * dirs[0], w.double() + step * dirs[1]) -
                    total(h.double() - step * dirs[0], w.double() - step * dirs[1])) / (2 * step)
            scale_of = float(((dh.double() * uh).abs().sum() if dirs[0].any() else (dw.double() * uw).abs().sum()))
            assert abs(float(got - diff)) < 1e-5 * scale_of


# ---------------------------------------------------------------- RMS norm

RMS_SHAPES = [(1, 8), (3, 64), (9, 72), (17, 128), (33, 136), (5, 256), (130, 264), (77, 512), (4, 520), (41, 1024),
              (2, 1032), (7, 1544), (300, 2560), (6, 2568), (5, 4104), (3, 8200), (2, 16384), (3, 16392), (2, 32768),
              (1, 32760)]
RMS_MANY = [(70000, 64), (30011, 256), (9001, 512), (2600, 2560), (1100, 5000), (700, 9000)]


def rms_sums(d):
    """Roundings of a row's sum: a lane's steps of eight, the lanes and the waves, 16 at most of each."""
    return 8 * 5 + 6 + 16


def rms_ref(x, res, gamma, eps, dtype):
    s = x if res is None else (x.float() + res.float()).to(tdt(dtype))
    rr = (s.double().square().mean(1) + eps).rsqrt()
    return s, rr, s.double() * rr[:, None] * gamma.double()


def check_8bit(q, sc, y, rel):
    """q and sc are y in 8 bits, where y may be off by `rel` of its value before it is rounded."""
    rows, d = y.shape
    kb = -(-d // 128)
    q, sc, y = q.cpu().double(), sc.cpu().view(torch.uint8).to(torch.int64), y.cpu()
    assert (sc[:, kb:] == 127).all()
    top = torch.nn.functional.pad(y.abs(), (0, -d % 128)).reshape(rows, kb, 128).amax(2)
    exps = []
    for f in (1 - rel, 1 + rel):
        e = torch.ceil(torch.log2(top * f / 448.0)).clamp(min=-126)
        exps.append(torch.where(top > 0, e, torch.full_like(e, -126.0)).to(torch.int64) + 127)
    assert ((sc[:, :kb] == exps[0]) | (sc[:, :kb] == exps[1])).all()
    unit = torch.exp2((sc[:, :kb] - 127).double()).repeat_interleave(128, 1)[:, :d]
    # e4m3: half a step is 2^-4 of the value, 2^-10 below its normal range
    assert ((q * unit - y).abs() <= torch.maximum(2.0 ** -4 * y.abs() * (1 + rel), 2.0 ** -10 * unit) + rel * y.abs()).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", (True, False))
@pytest.mark.parametrize("rows,d", RMS_SHAPES + RMS_MANY)
def test_rms_norm(gpu, dtype, residual, rows, d):
    p = make_plan(dtype, d)
    x, gamma = randn((rows, d), dtype, 1).to(gpu), (1.0 + randn((d,), "f32", 2, 0.1)).to(gpu)
    res = randn((rows, d), dtype, 3, 2.0).to(gpu) if residual else None
    x[rows // 2] = 0.0
    if residual:
        res[rows // 2] = 0.0  # a row of padding
    total = nan_like(torch.empty_like(x)) if residual else None
    y, rr = nan_like(torch.empty_like(x)), nan_like(torch.empty(rows, device=gpu))
    q = torch.full((rows, d), 0x7F, dtype=torch.uint8, device=gpu).view(torch.float8_e4m3fn)
    sc = torch.full(p.fp8_scale_shape(rows, d, 1), 255, dtype=torch.uint8, device=gpu)
    p.engram_rms_norm(x, gamma, y, residual=res, total=total, q=q, scales=sc, rrms=rr, eps=1e-6)
    s, ref_rr, ref = rms_ref(x, res, gamma, 1e-6, dtype)
    if residual:
        assert torch.equal(total, s)
    rel = (rms_sums(d) / 2 + 6) * U
    close(rr, ref_rr.cpu(), rel * ref_rr.cpu(), "rrms")
    close(y, ref.cpu(), ((rel + 3 * U) + half_step(dtype) * 1.01) * ref.abs().cpu(), "y")
    check_8bit(q, sc, ref, rel + 3 * U)
    # each output alone is the same; the operator in 8 bits is its fp32 self quantised
    y2, q2, sc2 = torch.empty_like(y), torch.empty_like(q), torch.empty_like(sc)
    p.engram_rms_norm(x, gamma, y2, residual=res, total=total)
    p.engram_rms_norm(x, gamma, residual=res, total=total, q=q2, scales=sc2)
    assert torch.equal(y2, y) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(sc2, sc)
    if dtype == "f32":
        p.engram_quantize_fp8(y, q2, sc2)
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(sc2, sc)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,d", [(70, 64), (600, 136), (257, 1024), (66, 4104)])
def test_rms_norm_in_place(gpu, dtype, rows, d):
    p = make_plan(dtype, d)
    x, res, gamma = randn((rows, d), dtype, 1).to(gpu), randn((rows, d), dtype, 2).to(gpu), randn((d,), "f32", 3).to(gpu)
    total, y, rr = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=gpu)
    p.engram_rms_norm(x, gamma, y, residual=res, total=total, rrms=rr)
    for t_at, y_at in ((0, 1), (1, 0), (0, None), (1, None), (None, 0), (None, 1)):
        bufs = [x.clone(), res.clone()]
        t = bufs[t_at] if t_at is not None else torch.empty_like(x)
        o = bufs[y_at] if y_at is not None else torch.empty_like(x)
        p.engram_rms_norm(bufs[0], gamma, o, residual=bufs[1], total=t)
        assert torch.equal(t, total) and torch.equal(o, y)
    alone = x.clone()
    p.engram_rms_norm(alone, gamma, alone)
    p.engram_rms_norm(x, gamma, y)
    assert torch.equal(alone, y)
    # x twice: the sum of a row with itself
    p.engram_rms_norm(x, gamma, y, residual=x, total=total)
    assert torch.equal(total, (x.float() + x.float()).to(x.dtype))
    # the backward in place of each of its inputs
    dy, dt = randn((rows, d), dtype, 4).to(gpu), randn((rows, d), dtype, 5).to(gpu)
    p.engram_rms_norm(x, gamma, y, residual=res, total=total, rrms=rr)
    ws, dg, dx = p.rms_norm_backward_workspace(rows), torch.empty(d, device=gpu), torch.empty_like(x)
    p.engram_rms_norm_backward(total, dy, gamma, rr, dx, dg, ws, dtotal=dt)
    for at in range(3):
        b = [total.clone(), dy.clone(), dt.clone()]
        dg2 = torch.empty_like(dg)
        p.engram_rms_norm_backward(b[0], b[1], gamma, rr, b[at], dg2, ws, dtotal=b[2])
        assert torch.equal(b[at], dx) and torch.equal(dg2, dg)


def test_rms_norm_rows_are_apart(gpu):
    """An infinity, a NaN or the type's largest values in a row change no other row."""
    for d in (64, 128, 256, 1024, 4104):
        p = make_plan("bf16", d)
        x, gamma = randn((70, d), "bf16", 1).to(gpu), torch.ones(d, device=gpu)
        sc_shape = p.fp8_scale_shape(70, d, 1)

        def call(x):
            y, q, sc = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=gpu), \
                torch.empty(sc_shape, dtype=torch.uint8, device=gpu)
            p.engram_rms_norm(x, gamma, y, q=q, scales=sc)
            return y, q.view(torch.uint8), sc

        clean = call(x)
        bad = x.clone()
        bad[5, 3], bad[9, d - 1], bad[33, 0], bad[40] = math.inf, math.nan, -math.inf, torch.finfo(torch.bfloat16).max
        got = call(bad)
        ok = torch.ones(70, dtype=torch.bool, device=gpu)
        ok[[5, 9, 33, 40]] = False
        for a, b in zip(clean, got):
            assert torch.equal(a[ok], b[ok])
        assert got[0][9].isnan().all() and got[0][5, 3].isnan() and (got[0][5, :3] == 0).all()
        assert ((got[1][9] & 0x7F) == 0x7F).all() and int(got[1][5, 3]) & 0x7F == 0x7F


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", (True, False))
@pytest.mark.parametrize("rows,d", RMS_SHAPES + RMS_MANY)
def test_rms_norm_backward(gpu, dtype, residual, rows, d):
    p = make_plan(dtype, d)
    s, dy = randn((rows, d), dtype, 1).to(gpu), randn((rows, d), dtype, 2).to(gpu)
    gamma = (1.0 + randn((d,), "f32", 3, 0.1)).to(gpu)
    dt = randn((rows, d), dtype, 4).to(gpu) if residual else None
    rr = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dg = nan_like(torch.empty_like(s)), nan_like(torch.empty(d, device=gpu))
    ws = p.rms_norm_backward_workspace(rows)
    ws.fill_(255)
    p.engram_rms_norm_backward(s, dy, gamma, rr, dx, dg, ws, dtotal=dt)
    r, xh = rr.double()[:, None], s.double() * rr.double()[:, None]
    g = dy.double() * gamma.double()
    m = (g * xh).mean(1, keepdim=True)
    ref = r * (g - xh * m) + (0 if dt is None else dt.double())
    mag_m = (g * xh).abs().mean(1, keepdim=True)
    off = r * (3 * U * g.abs() + xh.abs() * ((rms_sums(d) + 8) * U * mag_m)) + 4 * U * ref.abs() + half_step(dtype) * ref.abs()
    off = off + 4 * U * (r * (g.abs() + (xh * m).abs()))
    close(dx, ref.cpu(), off.cpu(), "dx")
    # a lane's rows, the blocks' parts by 16 waves
    n_sum = rows / 64 + 200
    ref_g, mag_g = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    close(dg, ref_g.cpu(), ((min(rows, n_sum) + 4) * U * mag_g).cpu(), "dgamma")
    before = randn((d,), "f32", 6).to(gpu)
    acc = before.clone()
    p.engram_rms_norm_backward(s, dy, gamma, rr, dx, acc, ws, dtotal=dt, flags=8)
    assert torch.equal(acc, before + dg)


def test_rms_norm_backward_is_the_difference_of_the_norm(gpu):
    rows, d, eps = 7, 264, 1e-6
    p = make_plan("f32", d)
    x, dy, gamma = randn((rows, d), "f32", 1).to(gpu), randn((rows, d), "f32", 2).to(gpu), randn((d,), "f32", 3).to(gpu)
    y, rr = torch.empty_like(x), torch.empty(rows, device=gpu)
    p.engram_rms_norm(x, gamma, y, rrms=rr, eps=eps)
    dx, dg = torch.empty_like(x), torch.empty(d, device=gpu)
    p.engram_rms_norm_backward(x, dy, gamma, rr, dx, dg, p.rms_norm_backward_workspace(rows))

    def total(xx, gg):
        return (dy.double() * xx * (xx.square().mean(1, keepdim=True) + eps).rsqrt() * gg).sum()

    for seed in range(4):
        ux, ug = randn((rows, d), "f32", 20 + seed).to(gpu).double(), randn((d,), "f32", 30 + seed).to(gpu).double()
        step = 1e-4
        for a, b, got, mag in ((ux, 0 * ug, (dx.double() * ux).sum(), (dx.double() * ux).abs().sum()),
                               (0 * ux, ug, (dg.double() * ug).sum(), (dg.double() * ug).abs().sum())):
            diff = (total(x.double() + step * a, gamma.double() + step * b) -
                    total(x.double() - step * a, gamma.double() - step * b)) / (2 * step)
            assert abs(float(got - diff)) < 1e-5 * float(mag)


# ---------------------------------------------------------------- clipping


def grads_of(sizes, dtypes, seed, gpu, sd=1.0):
    return [(torch.randn(n, generator=gen(seed + i)) * sd * 10.0 ** (i % 3 - 1)).to(tdt(t)).to(gpu)
            for i, (n, t) in enumerate(zip(sizes, dtypes))]


def norm_ref(grads, counts=None):
    total = 0.0
    for i, g in enumerate(grads):
        x = g.double().cpu()
        if counts is not None and counts[i] is not None:
            x = torch.cat([x[k, :max(0, min(int(c), x.shape[1]))].flatten() for k, c in enumerate(counts[i])])
        total += float(x.square().sum())
    return math.sqrt(total)


def check_clip(p, B, grads, max_norm, counts=None, in_place=False):
    outs = None if in_place else [torch.full_like(g, 5.0) for g in grads]
    before = [g.clone() for g in grads]
    lst = B.GradList(grads, outs=outs, row_counts=counts)
    norm = nan_like(torch.empty(2, device=grads[0].device))
    p.engram_clip_grads(lst, norm, p.clip_grads_workspace(lst), max_norm=max_norm)
    ref = norm_ref(before, counts)
    n, f = norm.tolist()
    assert abs(n - ref) <= 1.01 * U * ref
    top = float(torch.tensor(max_norm, dtype=torch.float32))  # the argument is an fp32 number: 1e-3 is off by up to u
    want = top / ref if ref > top else 1.0
    assert abs(f - want) <= 1.01 * U * want
    for i, (b, o) in enumerate(zip(before, grads if in_place else outs)):
        exp = (b.float() * torch.tensor(f, dtype=torch.float32, device=b.device)).to(b.dtype)
        if counts is not None and counts[i] is not None:
            rest = b if in_place else torch.full_like(b, 5.0)
            live = torch.arange(b.shape[1], device=b.device)[None, :] < counts[i][:, None]
            exp = torch.where(live.reshape(live.shape + (1,) * (b.dim() - 2)), exp, rest)
        assert torch.equal(o, exp), i
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))


@pytest.mark.parametrize("in_place", (False, True))
@pytest.mark.parametrize("max_norm", (1e-3, 1.0, 1e30, math.inf))
@pytest.mark.parametrize("sizes", [(1,), (7, 8, 9), (0, 5, 0), (8191, 8192, 8193, 0), (100003, 1, 33, 4097),
                                   tuple(range(1, 130)), (20_000_001, 17, 3_000_000)])
def test_clip_grads(gpu, in_place, max_norm, sizes):
    from hashed_gram_embedding_vocab_amd import binding as B

    dtypes = ["bf16" if i % 3 == 1 else "f32" for i in range(len(sizes))]
    check_clip(make_plan(), B, grads_of(sizes, dtypes, 3, gpu), max_norm, in_place=in_place)


@pytest.mark.parametrize("in_place", (False, True))
@pytest.mark.parametrize("groups,rows,tail", [(1, 1, (1,)), (3, 5, (7,)), (8, 333, (32,)), (2, 3000, (4, 3)), (16, 1, (8,)), (5, 40, ())])
def test_clip_grads_takes_the_first_rows_of_a_group(gpu, in_place, groups, rows, tail):
    from hashed_gram_embedding_vocab_amd import binding as B

    for dtype in DTYPES:
        g = randn((groups, rows) + tail, dtype, 1).to(gpu)
        counts = torch.randint(-2, rows + 3, (groups,), generator=gen(2)).to(torch.int32)
        counts[0], counts[-1] = 0, rows
        counts = counts.to(gpu)
        for k in range(groups):  # what takes no part may hold anything
            g[k, max(0, int(counts[k])):] = 3e38
        plain = randn((1001,), "f32", 3).to(gpu)
        check_clip(make_plan(), B, [g, plain], 0.5, counts=[counts, None], in_place=in_place)


def test_clip_grads_norms_of_every_size(gpu):
    """Squares below and above fp32's range, and norms that are not finite."""
    from hashed_gram_embedding_vocab_amd import binding as B

    p = make_plan()
    norm = torch.empty(2, device=gpu)
    for v in (1e-38, 1e-30, 1e30, 3e38):
        g = torch.full((1000,), v, device=gpu)
        lst = B.GradList([g], outs=[torch.empty_like(g)])
        p.engram_clip_grads(lst, norm, p.clip_grads_workspace(1), max_norm=1.0)
        ref = float(g[0].double()) * math.sqrt(1000)
        n, f = norm.tolist()
        assert (abs(n - ref) <= 1.01 * U * ref) if ref < 3.4e38 else n == math.inf
        assert abs(f - min(1.0, 1.0 / ref)) <= 1.01 * U * f + 2.0 ** -149
    for v in (math.inf, -math.inf, math.nan):
        g = torch.ones(5000, device=gpu)
        g[4321] = v
        keep = g.clone()
        out = torch.zeros_like(g)
        p.engram_clip_grads(B.GradList([g]), norm, p.clip_grads_workspace(1), max_norm=1.0)
        p.engram_clip_grads(B.GradList([g], outs=[out]), norm, p.clip_grads_workspace(1), max_norm=1.0)
        n, f = norm.tolist()
        assert not math.isfinite(n) and f == 1.0
        for t in (g, out):
            assert torch.equal(t.nan_to_num(9.0, 8.0, 7.0), keep.nan_to_num(9.0, 8.0, 7.0))
    g = torch.zeros(77, device=gpu)
    p.engram_clip_grads(B.GradList([g]), norm, p.clip_grads_workspace(1), max_norm=1.0)
    assert norm.tolist() == [0.0, 1.0]
    g = torch.ones(77, device=gpu)  # only the norm is wanted
    p.engram_clip_grads(B.GradList([g], outs=[None]), norm, p.clip_grads_workspace(1), max_norm=0.5)
    assert abs(float(norm[0]) - math.sqrt(77)) < 1e-6 and (g == 1).all()


# ---------------------------------------------------------------- together, streams, graphs


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok,vocab,d", [(1, 1, 8), (45, 37, 72), (300, 333, 264), (700, 1111, 520), (1030, 16500, 72),
                                           (131, 50, 2568), (4100, 70, 136)])
def test_nothing_is_written_beside_the_outputs(gpu, dtype, n_tok, vocab, d):
    """Every output and workspace with bytes around it, at sizes that end inside a
    vector, a block, a tile and a word of scales."""
    from hashed_gram_embedding_vocab_amd import binding as B

    p = make_plan(dtype, d, vocab)
    dt, f32, u8 = tdt(dtype), torch.float32, torch.uint8
    made = []

    def buf(shape, t):
        made.append(Guarded(shape, t, gpu))
        return made[-1].t

    h, w, y = head(dtype, n_tok, vocab, d, 1.0, 3, gpu)
    gamma = 1.0 + randn((d,), "f32", 3, 0.1).to(gpu)
    total, yn, rr = buf((n_tok, d), dt), buf((n_tok, d), dt), buf((n_tok,), f32)
    p.engram_rms_norm(h, gamma, yn, residual=h, total=total, q=buf((n_tok, d), torch.float8_e4m3fn),
                      scales=buf(p.fp8_scale_shape(n_tok, d, 1), u8), rrms=rr)
    dg = buf((d,), f32)
    p.engram_rms_norm_backward(total, yn, gamma, rr, buf((n_tok, d), dt), dg,
                               buf((p.engram_rms_norm_backward_workspace_size(n_tok),), u8), dtotal=h)
    loss, lse = buf((n_tok,), f32), buf((n_tok,), f32)
    p.engram_cross_entropy(h, w, y, loss, lse, buf((p.engram_cross_entropy_workspace_size(n_tok),), u8))
    outs = []
    for dw_dtype in (f32, torch.bfloat16) if dtype == "bf16" else (f32,):
        ws = buf((p.engram_cross_entropy_backward_workspace_size(n_tok, dw_dtype),), u8)
        outs += [buf((n_tok, d), dt), buf((vocab, d), dw_dtype)]
        p.engram_cross_entropy_backward(h, w, y, lse, None, outs[-2], outs[-1], ws)
    counts = torch.tensor([0, n_tok, n_tok // 2], dtype=torch.int32, device=gpu)
    rows = randn((3, n_tok, 7), "f32", 5).to(gpu)
    grads, row_counts = outs + [dg, rows, rows[0, 0].clone()], [None] * (len(outs) + 1) + [counts, None]
    lst = B.GradList(grads, outs=[buf(tuple(g.shape), g.dtype) for g in grads], row_counts=row_counts)
    p.engram_clip_grads(lst, buf((2,), f32), buf((p.engram_clip_grads_workspace_size(len(grads)),), u8), max_norm=1e-3)
    torch.cuda.synchronize()
    assert all(g.whole() for g in made), [i for i, g in enumerate(made) if not g.whole()]


def test_a_training_step_through_all_of_them(gpu):
    """Tokens -> tied embedding -> residual and RMS norm in 8 bits -> a projection ->
    residual and norm -> loss, and back, the tied table's gradient from both ends in
    one buffer, clipped together.  Every stage against 64 bits on what the stage
    before gave."""
    from hashed_gram_embedding_vocab_amd import binding as B

    n, V, d = 300, 1111, 264
    p = make_plan("bf16", d, V)
    bf, f32 = dict(dtype=torch.bfloat16, device=gpu), dict(dtype=torch.float32, device=gpu)
    ids, targets = zipf_ids(n, V, 1).to(gpu), zipf_ids(n, V, 2).to(gpu)
    table, gamma1, gamma2 = randn((V, d), "bf16", 3, 0.3).to(gpu), torch.ones(d, **f32), 1.0 + randn((d,), "f32", 4, 0.1).to(gpu)
    wp = randn((d, d), "bf16", 5, 0.05).to(gpu)
    h0, x1, t2, y2 = (torch.empty((n, d), **bf) for _ in range(4))
    p.engram_embed(ids, table, h0.view(1, n, d))
    q, sc = torch.empty((n, d), dtype=torch.float8_e4m3fn, device=gpu), torch.empty(p.fp8_scale_shape(n, d, 1), dtype=torch.uint8, device=gpu)
    rr1, rr2 = torch.empty(n, **f32), torch.empty(n, **f32)
    y1 = torch.empty((n, d), **bf)
    p.engram_rms_norm(h0, gamma1, y1, q=q, scales=sc, rrms=rr1)
    kp = 272  # (a product's K is a multiple of 16)
    qp, sp = torch.zeros((n, kp), dtype=torch.uint8, device=gpu), sc
    qp[:, :d] = q.view(torch.uint8)
    wq, ws8 = torch.empty((d, kp), dtype=torch.float8_e4m3fn, device=gpu), torch.empty(p.fp8_scale_shape(d, kp, 128), dtype=torch.uint8, device=gpu)
    p.engram_quantize_fp8(torch.nn.functional.pad(wp, (0, kp - d)), wq, ws8, block_rows=128)
    p.engram_matmul_fp8(qp.view(torch.float8_e4m3fn), sp, wq, ws8, x1, p.matmul_fp8_workspace(n, d, kp))
    p.engram_rms_norm(x1, gamma2, y2, residual=h0, total=t2, rrms=rr2)
    s2, ref_rr, ref_y = rms_ref(x1, h0, gamma2, 1e-6, "bf16")
    assert torch.equal(t2, s2)
    close(y2, ref_y.cpu(), 2.0 ** -8 * 1.02 * ref_y.abs().cpu(), "y2")
    loss, lse = torch.empty(n, **f32), torch.empty(n, **f32)
    p.engram_cross_entropy(y2, table, targets, loss, lse, p.cross_entropy_workspace(n))
    ref = HeadRef(y2, table, targets, 1.0, "bf16")
    r = [t.cpu() for t in ref.forward()]
    close(loss, r[0], r[2], "loss")
    counted = int(ref.counts.sum())
    dy2, dtable = torch.empty((n, d), **bf), torch.empty((V, d), **f32)
    p.engram_cross_entropy_backward(y2, table, targets, lse, None, dy2, dtable, p.cross_entropy_backward_workspace(n),
                                    dloss_scale=1.0 / counted)
    g = torch.full((n,), 1.0 / counted, dtype=torch.float64, device=gpu)
    rdh, off_h, rdw, off_w = (t.cpu() for t in ref.backward(lse, g, torch.float32))
    close(dy2, rdh, off_h, "dy2")
    close(dtable, rdw, off_w, "dtable, the head's part")
    dt2, dg2 = torch.empty((n, d), **bf), torch.empty(d, **f32)
    p.engram_rms_norm_backward(t2, dy2, gamma2, rr2, dt2, dg2, p.rms_norm_backward_workspace(n))
    # (the projection's own gradients go the way of the 8-bit product; here its input's is taken in 16 bits)
    dy1 = (dt2.float() @ wp.float()).to(torch.bfloat16)
    dh0, dg1 = torch.empty((n, d), **bf), torch.empty(d, **f32)
    p.engram_rms_norm_backward(h0, dy1, gamma1, rr1, dh0, dg1, p.rms_norm_backward_workspace(n), dtotal=dt2)
    head_part = dtable.clone()
    p.engram_embed_backward(ids, dh0.view(1, n, d), dtable, p.embed_backward_workspace(n), flags=B.GRAD_ACCUMULATE)
    ok = (ids >= 0) & (ids < V)
    both = head_part.double().index_add_(0, ids[ok].long(), dh0.double()[ok])
    mag = head_part.double().abs().index_add_(0, ids[ok].long(), dh0.double().abs()[ok])
    close(dtable, both.cpu(), (n * U * mag).cpu(), "dtable")
    lst = B.GradList([dtable, dg1, dg2])
    norm = torch.empty(2, **f32)
    before = [t.clone() for t in lst.grads]
    ref_norm = norm_ref(before)
    p.engram_clip_grads(lst, norm, p.clip_grads_workspace(lst), max_norm=0.5 * ref_norm)
    assert abs(float(norm[0]) - ref_norm) <= 1.01 * U * ref_norm and abs(float(norm[1]) - 0.5) <= 4 * U
    assert all(torch.equal(a, b * norm[1]) for a, b in zip(lst.grads, before))
    assert abs(norm_ref(lst.grads) - 0.5 * ref_norm) <= 1e-6 * ref_norm


def _ends(gpu, seed, n, V=1030, d=136, dw_dtype=torch.float32):
    """A call of every operator on buffers of its own."""
    from hashed_gram_embedding_vocab_amd import binding as B

    p = make_plan("bf16", d, V)
    h, w, y = head("bf16", n, V, d, 1.0, seed, gpu)
    gamma = 1.0 + randn((d,), "f32", seed, 0.1).to(gpu)
    e = torch.empty_like
    total, yn, dx, dh = e(h), e(h), e(h), e(h)
    q, sc = torch.empty(h.shape, dtype=torch.float8_e4m3fn, device=gpu), torch.empty(p.fp8_scale_shape(n, d, 1), dtype=torch.uint8, device=gpu)
    rr, loss, lse = (torch.empty(n, device=gpu) for _ in range(3))
    dg, dw = torch.empty(d, device=gpu), torch.empty((V, d), dtype=dw_dtype, device=gpu)
    rows, counts = randn((4, 50, 16), "f32", seed).to(gpu), torch.tensor([0, 50, 7, 21], dtype=torch.int32, device=gpu)
    ro = torch.zeros_like(rows)
    outs = [e(dg), e(dw), ro]
    lst = B.GradList([dg, dw, rows], outs=outs, row_counts=[None, None, counts])
    norm = torch.empty(2, device=gpu)
    ws = (p.rms_norm_backward_workspace(n), p.cross_entropy_workspace(n), p.cross_entropy_backward_workspace(n, dw_dtype),
          p.clip_grads_workspace(lst))

    def call(stream=None):
        p.engram_rms_norm(h, gamma, yn, residual=h, total=total, q=q, scales=sc, rrms=rr, stream=stream)
        p.engram_cross_entropy(yn, w, y, loss, lse, ws[1], stream=stream)
        p.engram_cross_entropy_backward(yn, w, y, lse, None, dh, dw, ws[2], stream=stream)
        p.engram_rms_norm_backward(total, dh, gamma, rr, dx, dg, ws[0], dtotal=dh, stream=stream)
        p.engram_clip_grads(lst, norm, ws[3], max_norm=0.01, stream=stream)

    return call, [total, yn, q.view(torch.uint8), sc, rr, loss, lse, dh, dw, dx, dg, norm] + outs, y


def test_captured_graphs_replay_the_eager_results(gpu):
    """Two graphs with workspaces of their own, replayed several times and at once
    on two streams, with eager work in between and inputs changed."""
    sets = [_ends(gpu, 60, 700), _ends(gpu, 70, 33, dw_dtype=torch.bfloat16)]
    eager = []
    for call, outs, _ in sets:
        call()
        torch.cuda.synchronize()
        eager.append([o.clone() for o in outs])
    graphs = []
    for call, outs, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for turn in range(4):
        for _, outs, _ in sets:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (_, outs, _), want in zip(sets, eager):
            for o, e in zip(outs, want):
                assert torch.equal(o, e), turn
        sets[0][0]()  # eager work between the replays
    sets[0][2].copy_(zipf_ids(700, 1030, 99).to(gpu))
    graphs[0].replay()
    torch.cuda.synchronize()
    replayed = [o.clone() for o in sets[0][1]]
    sets[0][0]()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, sets[0][1]))
    assert not torch.equal(replayed[5], eager[0][5])


def test_side_stream(gpu):
    """On a stream of the caller's, behind work of that stream, without touching the current one."""
    call, outs, y = _ends(gpu, 80, 700)
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    keep = y.clone()
    y.fill_(0)
    for o in outs:
        o.zero_()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        big = torch.zeros(1 << 28, device=gpu)  # work the calls have to wait behind
        big += 1
        y.copy_(keep)
    call(st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_profiling_counts_the_operators(gpu):
    call, _, _ = _ends(gpu, 90, 40)
    p = call.__closure__  # (a plan of its own would count the same; the call's is used below)
    from hashed_gram_embedding_vocab_amd import binding as B

    plan = [c.cell_contents for c in p if isinstance(c.cell_contents, B.Plan)][0]
    call()
    plan.engram_profile_begin(16)
    call()
    r = plan.engram_profile_end()
    assert r["aux"]["launches"] == 2 and r["gemm"]["launches"] == 1 and r["bwd_gemm"]["launches"] == 1
    assert r["bwd_fuse"]["launches"] == 1 and r["bwd_gemm"]["total_ms"] > 0


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
@pytest.mark.parametrize("n_tok", (1, 3, 21, 33, 64, 65, 200, 700, 4100))
@pytest.mark.parametrize("vocab,d", [(5, 8), (300, 72), (1000, 264), (5003, 136), (40000, 64), (2000, 2560)])
def test_accumulated_weight_gradients_are_rounded_once(gpu, dtype, dw_dtype, n_tok, vocab, d):
    """What is there plus the increment in fp32, rounded once, however the sums are split.
    An lse of 1000 beside logits of 0 leaves P = -g at the target and 0 elsewhere; h's and
    g's few bits make each increment, and its sum with the old value, exact in fp32."""
    p = make_plan(dtype, d, vocab)
    h = (torch.randint(-255, 256, (n_tok, d), generator=gen(1)) / 64.0).to(tdt(dtype)).to(gpu)
    w = torch.zeros((vocab, d), dtype=tdt(dtype), device=gpu)
    y = (torch.arange(n_tok, device=gpu) % min(vocab, 7) * (vocab // 7 + 1) % vocab).to(torch.int32)
    g = 2.0 ** torch.randint(-2, 2, (n_tok,), generator=gen(2)).to(gpu)
    lse = torch.full((n_tok,), 1000.0, device=gpu)
    # (bf16: 8 bits of 2^-8 and more)
    old = (torch.randint(-255, 256, (vocab, d), generator=gen(3)) / 256.0).to(dw_dtype).to(gpu)
    inc = torch.zeros((vocab, d), dtype=torch.float64, device=gpu).index_add_(0, y.long(), -g.double()[:, None] * h.double())
    want = (old.double() + inc).float()
    assert torch.equal(want.double(), old.double() + inc)
    ws = p.cross_entropy_backward_workspace(n_tok, dw_dtype)
    for dh in (None, torch.empty_like(h)):
        dw = old.clone()
        p.engram_cross_entropy_backward(h, w, y, lse, g, dh, dw, ws, flags=8)
        assert torch.equal(dw, want.to(dw_dtype))


@pytest.mark.parametrize("n_tok,vocab,d", [(1030, 16500, 128), (4100, 300, 192), (12290, 270, 64), (4100, 1000, 320)])
def test_rows_of_whole_lines_are_read_where_they_are(gpu, n_tok, vocab, d):
    """Token counts from which rows that are no whole lines are copied into blocks first."""
    p = make_plan("bf16", d, vocab)
    h, w, y = head("bf16", n_tok, vocab, d, 1.0, 3, gpu)
    loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
    p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok))
    ref, ref_lse, off, off_lse = (t.cpu() for t in HeadRef(h, w, y, 1.0, "bf16").forward())
    close(loss, ref, off, "loss")
    close(lse, ref_lse, off_lse, "lse")
    for dw_dtype in (torch.bfloat16, torch.float32):
        check_backward(gpu, "bf16", dw_dtype, n_tok, vocab, d, 1.0)


@pytest.mark.parametrize("dtype,dw_dtype", GRADS)
@pytest.mark.parametrize("n_tok,vocab,d", PATHS)
def test_factors_whose_product_passes_fp32s_range(gpu, dtype, dw_dtype, n_tok, vocab, d):
    """g_t scale = dloss_t dloss_scale scale counts as a whole: 2^140 and 2^-160 as the last
    two's product, with the dloss that brings the whole back, give the bits of the same
    whole made of ordinary factors, and a token whose dloss is 0 has no part."""
    p = make_plan(dtype, d, vocab)
    r = torch.rand(n_tok, generator=gen(8)).to(gpu) + 0.1
    r[::3] = 0.0
    y = zipf_ids(n_tok, vocab, 3, bad=False).to(gpu)
    lse = torch.full((n_tok,), math.log(vocab), device=gpu)
    ws = p.cross_entropy_backward_workspace(n_tok, dw_dtype)
    for scale, loss_scale, dloss in ((2.0 ** 40, 2.0 ** 100, r * 2.0 ** -120), (2.0 ** -60, 2.0 ** -100, r * 2.0 ** 120)):
        h, w = randn((n_tok, d), dtype, 1).to(gpu), randn((vocab, d), dtype, 2, 2.0 ** -42 / math.sqrt(d)).to(gpu)
        results = []
        for s, g in ((loss_scale, dloss), (1.0, dloss.double() * loss_scale)):
            dh, dw = nan_like(torch.empty_like(h)), nan_like(torch.empty((vocab, d), dtype=dw_dtype, device=gpu))
            p.engram_cross_entropy_backward(h, w, y, lse, g.float(), dh, dw, ws, scale=scale, dloss_scale=s)
            results.append((dh, dw))
        assert all(torch.equal(a, b) for a, b in zip(*results))
        dh, dw = results[0]
        assert torch.isfinite(dh).all() and torch.isfinite(dw).all() and dw.count_nonzero()
        assert not dh[r == 0].count_nonzero()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sign", (1, -1))
def test_the_largest_scale(gpu, dtype, sign):
    """2^127 over weights of 2^-126: every product and sum is a normal number."""
    for n_tok, vocab, d in PATHS:
        p = make_plan(dtype, d, vocab)
        h = torch.randint(0, 4, (n_tok, d), generator=gen(1)).to(tdt(dtype)).to(gpu)
        w = (torch.randint(-1, 2, (vocab, d), generator=gen(2)) * 2.0 ** -126).to(tdt(dtype)).to(gpu)
        y = zipf_ids(n_tok, vocab, 3).to(gpu)
        loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
        p.engram_cross_entropy(h, w, y, loss, lse, p.cross_entropy_workspace(n_tok), scale=sign * 2.0 ** 127)
        ref, ref_lse, off, off_lse = (t.cpu() for t in HeadRef(h, w, y, sign * 2.0 ** 127, dtype).forward())
        close(loss, ref, off, "loss")
        close(lse, ref_lse, off_lse, "lse")


@pytest.mark.parametrize("n_tok,vocab,d", [(80, 129280, 64), (66, 40001, 72), (192, 40130, 6744)])
def test_the_tiles_sums_stay_in_their_region(gpu, n_tok, vocab, d):
    """fp32: more tiles of 64 x 64 than a launch of a smaller kind may have, and such tiles in
    two pieces of the vocabulary.  The logits of a few tokens, which these calls do not
    make, have the next region: it and what lies behind the workspace stay as they were."""
    p = make_plan("f32", d, vocab)
    h, w, y = head("f32", n_tok, vocab, d, 1.0, 3, gpu)
    loss, lse = nan_like(torch.empty(n_tok, device=gpu)), nan_like(torch.empty(n_tok, device=gpu))
    size = p.engram_cross_entropy_workspace_size(n_tok)
    ws = Guarded((size,), torch.uint8, gpu)
    ws.t.fill_(0x5A)
    p.engram_cross_entropy(h, w, y, loss, lse, ws.t)
    ref, ref_lse, off, off_lse = (t.cpu() for t in HeadRef(h, w, y, 1.0, "f32").forward())
    close(loss, ref, off, "loss")
    close(lse, ref_lse, off_lse, "lse")
    assert ws.whole()
    # targets' logits, then 2 ceil(V / 64) pairs a token at most, then 32 MB at most
    at = -(-4 * n_tok // 256) * 256 + -(-8 * 2 * -(-vocab // 64) * n_tok // 256) * 256
    few = min(32 << 20, 64 * n_tok * -(-vocab // 8) * 8 * 4)
    assert (ws.t[at:at + few] == 0x5A).all()
