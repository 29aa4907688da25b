"""The operators at a model's ends as measured cases: the output head's softmax
cross entropy with its gradients, RMS norm with the residual's addition (in 16,
32 or 8 bits) with its gradients, and the clipping of many gradients by their
common norm.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, through the
library's entry points.  ``exact`` gives the same outputs from the definitions
in 64 bits.

The definitions:

  loss       x[t][v] = scale <h_t, W_v>, lse_t = log sum_v exp x[t][v],
             loss_t = lse_t - x[t][y_t]; a target outside [0, vocab) gives
             loss_t = lse_t = 0
  loss_grad  P[t][v] = g_t scale (exp(x[t][v] - lse_t) - [v = y_t]) with g_t the
             loss's gradient (0 for such a target): dh = P W, dW = P^T h over
             the tokens that count
  norm       s = x + r rounded to the plan's type (s = x where there is no r),
             rr = (mean(s^2) + eps)^(-1/2), y = s rr gamma; in 8 bits: per 128
             values of a row the smallest power of two sc >= 2^-126 with
             amax / sc <= 448, q = y / sc rounded to e4m3
  norm_grad  g = dy gamma, x' = s rr:
             dx = rr (g - x' mean(g x')) + ds, dgamma = sum dy x'
  clip       norm = (sum of all tensors' x^2)^(1/2), c = max_norm / norm where
             that is below 1, else 1; out = c x.  Of each table's row gradients
             the first take part, as many as its count on the device says.
"""

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN_EXP = -126
EPS = 1e-6


def listed():
    return [
        # the log-probability of one sampled token
        dict(name="loss_one_token", op="loss", dtype="bf16", vocab=129280, d=2560, tokens=1, scale=1.0),
        # evaluation of one ragged sequence by a model in fp32
        dict(name="loss_f32", op="loss", dtype="f32", vocab=32000, d=1024, tokens=517, scale=1.0),
        # evaluation of a batch of 2 x 4096 tokens
        dict(name="loss_eval", op="loss", dtype="bf16", vocab=129280, d=2560, tokens=8192, scale=1.0),
        # fine-tuning on one short ragged batch in fp32
        dict(name="loss_grad_short", op="loss_grad", dtype="f32", vocab=1000, d=256, tokens=333, scale=0.0625, dw="f32"),
        # a micro-batch whose weight gradient is kept in fp32, as the tied embedding's is
        dict(name="loss_grad_f32_weight", op="loss_grad", dtype="bf16", vocab=32000, d=1024, tokens=4096, scale=1.0, dw="f32"),
        # the training step of 2 x 4096 tokens
        dict(name="loss_grad_train", op="loss_grad", dtype="bf16", vocab=129280, d=2560, tokens=8192, scale=1.0, dw="bf16"),
        # a decode step of 256 sequences: residual added, the 8-bit projection's input written
        dict(name="norm_decode_8bit", op="norm", dtype="bf16", d=2560, rows=256, residual=True, out="8bit"),
        # a prefill chunk of 8 x 4096 tokens, in both forms (8 bits for the projections, 16 for the rest)
        dict(name="norm_prefill_both", op="norm", dtype="bf16", d=2560, rows=32768, residual=True, out="both"),
        # the gradients of one short sequence in fp32, no residual
        dict(name="norm_grad_short", op="norm_grad", dtype="f32", d=1024, rows=517, residual=False),
        # the gradients of four branches of 32,768 tokens, with the residual stream's gradient
        dict(name="norm_grad_train", op="norm_grad", dtype="bf16", d=2560, rows=131072, residual=True),
        # one small layer's gradients: a dozen tensors, some of odd length
        dict(name="clip_small", op="clip", dtype="f32", vocab=1000, d=256, n_layers=1, table_rows=500, head_dim=32),
        # a model's: the embedding's table, four layers' projections and norms, their tables' rows
        dict(name="clip_model", op="clip", dtype="f32", vocab=129280, d=2560, n_layers=4, table_rows=32768, head_dim=80),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    return step * _log_int(rng, max(1, lo // step), hi // step)


def draw(rng):
    op = rng.choice(["loss", "loss", "loss_grad", "loss_grad", "norm", "norm_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    elem = 2 if dtype == "bf16" else 4
    while True:
        if op in ("loss", "loss_grad"):
            c = dict(op=op, dtype=dtype, vocab=_log_int(rng, 50, 200000), d=_width(rng, 64, 8192, 8),
                     tokens=_log_int(rng, 1, 8192), scale=rng.choice([1.0, 0.5]))
            if op == "loss_grad":
                c["dw"] = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
            cost = c["tokens"] * c["vocab"] * c["d"]
            if (cost <= 8192 * 129280 * 2560 // 8 and c["vocab"] * c["d"] <= 129280 * 2560
                    and c["tokens"] * c["vocab"] <= 8192 * 129280):
                return c
        elif op in ("norm", "norm_grad"):
            c = dict(op=op, dtype=dtype, d=_width(rng, 64, 16384, 8), rows=_log_int(rng, 1, 131072),
                     residual=rng.random() < 0.7)
            if op == "norm":
                c["out"] = rng.choice(["same", "8bit", "both"])
            if c["rows"] * c["d"] * elem <= 131072 * 2560:
                return c
        else:
            c = dict(op=op, dtype=dtype, vocab=_log_int(rng, 50, 200000), d=_width(rng, 64, 8192, 8),
                     n_layers=rng.randint(1, 10), table_rows=_log_int(rng, 1, 32768), head_dim=_width(rng, 8, 256, 8))
            if sum(_clip_sizes(c)) <= sum(_clip_sizes(dict(vocab=129280, d=2560, n_layers=4, table_rows=32768, head_dim=80))):
                return c


# ---------------------------------------------------------------- inputs


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _randn(g, shape, dtype, sd=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * sd).to(dtype)


def _targets(g, n, vocab, s=1.05):
    """Zipf ids over a random rank-to-id order; one in twenty does not count (-1)."""
    w = torch.arange(1, vocab + 1, dtype=torch.float64, device="cuda").pow(-s).cumsum(0)
    u = torch.rand(n, dtype=torch.float64, device="cuda", generator=g) * w[-1]
    rank = torch.searchsorted(w, u).clamp_(max=vocab - 1)
    ids = torch.randperm(vocab, device="cuda", generator=g)[rank]
    skip = torch.rand(n, device="cuda", generator=g) < 0.05
    skip[0] = False
    return torch.where(skip, torch.full_like(ids, -1), ids).to(torch.int32)


def _activations(g, rows, d, dtype):
    """Hidden states: a common offset per channel and a few large channels."""
    gain = torch.where(torch.rand(d, device="cuda", generator=g) < 0.01, 12.0, 1.0)
    x = torch.randn((rows, d), device="cuda", generator=g)
    return (x * gain + 0.3 * torch.randn(d, device="cuda", generator=g)).to(dtype)


def _clip_sizes(c):
    """The gradients' sizes: the embedding, then each layer's projections (five of
    them), gammas, taps and its tables' rows."""
    d, k = c["d"], c["head_dim"] * 16
    layer = [5 * d * k, d, d, 4 * d, 3 * d + 1, 16 * c["table_rows"] * c["head_dim"]]
    return [c["vocab"] * d] + layer * c["n_layers"]


def _plan(case):
    from hashed_gram_embedding_vocab_amd import binding as B

    return B.Plan(vocab=case.get("vocab", 1000), vocab_comp=min(case.get("vocab", 1000), 770), heads=1, head_dim=128,
                  table_rows=[101, 103], hash_seed=1, d_model=case.get("d", 256),
                  dtype=B.F32 if case.get("dtype") == "f32" else B.BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, d = case["op"], case["d"]
    s = dict(case=dict(case))
    f32 = dict(dtype=torch.float32, device="cuda")
    if op in ("loss", "loss_grad"):
        dt, V, n = _dt(case["dtype"]), case["vocab"], case["tokens"]
        sd = 1.0 / math.sqrt(d) / case["scale"]
        s["w"] = w = _randn(g, (V, d), dt, sd)
        s["targets"] = y = _targets(g, n, V)
        # some tokens are nearly certain, some are guesses: logits of 0 to 12 at the target
        sure = 12.0 * torch.rand((n, 1), device="cuda", generator=g)
        h = torch.randn((n, d), device="cuda", generator=g)
        s["h"] = (h + sure * w[y.clamp(min=0).long()].float() / (sd * sd * d * case["scale"])).to(dt)
        s["lse"] = torch.empty(n, **f32)
        if op == "loss":
            s["loss"] = torch.empty(n, **f32)
        else:
            for i in range(0, n, 512):  # what the forward pass kept
                x = (s["h"][i:i + 512].float() @ w.float().t()).double() * case["scale"]
                s["lse"][i:i + 512] = torch.where(y[i:i + 512] >= 0, x.logsumexp(1), 0.0).float()
            count = (y >= 0).sum()
            s["dloss"] = (0.5 + torch.rand(n, device="cuda", generator=g)) / count
            s["dh"] = torch.empty_like(s["h"])
            s["dw"] = torch.empty((V, d), dtype=_dt(case["dw"]), device="cuda")
    elif op in ("norm", "norm_grad"):
        dt, rows = _dt(case["dtype"]), case["rows"]
        s["x"] = _activations(g, rows, d, dt)
        s["gamma"] = 1.0 + 0.1 * torch.randn(d, device="cuda", generator=g)
        if op == "norm":
            s["r"] = _activations(g, rows, d, dt) if case["residual"] else None
            s["total"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["rrms"] = torch.empty(rows, **f32)
            s["y"] = torch.empty_like(s["x"]) if case["out"] != "8bit" else None
            s["q"] = s["sc"] = None
            if case["out"] != "same":
                s["q"] = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device="cuda")
                s["sc"] = torch.empty((rows, -(-d // 512) * 4), dtype=torch.float8_e8m0fnu, device="cuda")
        else:
            s["dy"] = _randn(g, (rows, d), dt, 1e-2)
            s["ds"] = _randn(g, (rows, d), dt, 1e-2) if case["residual"] else None
            s["rrms"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(d, **f32)
    else:
        tensors, rows = [], []
        for i, n in enumerate(_clip_sizes(case)):
            j = (i - 1) % 6 if i else -1
            if j == 5:
                tensors.append(_randn(g, (16, case["table_rows"], case["head_dim"]), torch.float32, 1e-3))
                rows.append(torch.randint(0, case["table_rows"] + 1, (16,), device="cuda", generator=g).to(torch.int32))
            else:
                tensors.append(_randn(g, (n,), _dt(case["dtype"]) if j < 1 else torch.float32, 10.0 ** -(2 + i % 4)))
                rows.append(None)
        s["grads"], s["rows"] = tensors, rows
        s["outs"] = [torch.zeros_like(t) for t in tensors]
        s["norm"] = torch.empty(2, **f32)
        s["max_norm"] = 1.0
    if own:  # the plan, the workspace and the list of gradients that a program keeps
        from hashed_gram_embedding_vocab_amd import binding as B

        s["plan"] = p = _plan(case)
        if op == "loss":
            s["ws"] = p.cross_entropy_workspace(case["tokens"])
        elif op == "loss_grad":
            s["ws"] = p.cross_entropy_backward_workspace(case["tokens"], dweight_dtype=_dt(case["dw"]))
        elif op == "norm_grad":
            s["ws"] = p.rms_norm_backward_workspace(case["rows"])
        elif op == "clip":
            s["list"] = B.GradList(s["grads"], outs=s["outs"], row_counts=s["rows"])
            s["ws"] = p.clip_grads_workspace(s["list"])
    return s


# ---------------------------------------------------------------- the passes


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, p = s["case"], s["plan"]
    op = c["op"]
    if op == "loss":
        p.engram_cross_entropy(s["h"], s["w"], s["targets"], s["loss"], s["lse"], s["ws"], scale=c["scale"])
        return s["loss"], s["lse"]
    if op == "loss_grad":
        p.engram_cross_entropy_backward(s["h"], s["w"], s["targets"], s["lse"], s["dloss"], s["dh"], s["dw"], s["ws"],
                                        scale=c["scale"])
        return s["dh"], s["dw"]
    if op == "norm":
        p.engram_rms_norm(s["x"], s["gamma"], s["y"], residual=s["r"], total=s["total"], q=s["q"], scales=s["sc"],
                          rrms=s["rrms"], eps=EPS)
        return s["y"], s["total"], s["q"], s["sc"], s["rrms"]
    if op == "norm_grad":
        p.engram_rms_norm_backward(s["x"], s["dy"], s["gamma"], s["rrms"], s["dx"], s["dgamma"], s["ws"], dtotal=s["ds"])
        return s["dx"], s["dgamma"]
    p.engram_clip_grads(s["list"], s["norm"], s["ws"], max_norm=s["max_norm"])
    return s["norm"], s["outs"]


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("loss", "loss_grad"):
        h, w, y = s["h"].float(), s["w"].float(), s["targets"].long()
        counts, at = y >= 0, y.clamp(min=0)[:, None]
        x = h @ w.t()
        if c["scale"] != 1.0:
            x *= c["scale"]
        if op == "loss":
            top = x.amax(1, keepdim=True)
            lse = (x - top).exp_().sum(1).log() + top[:, 0]
            zero = torch.zeros_like(lse)
            return torch.where(counts, lse - x.gather(1, at)[:, 0], zero), torch.where(counts, lse, zero)
        p = x.sub_(s["lse"][:, None]).exp_()
        p.scatter_(1, at, p.gather(1, at) - 1.0)
        p *= (torch.where(counts, s["dloss"], torch.zeros_like(s["dloss"])) * c["scale"])[:, None]
        return (p @ w).to(s["h"].dtype), (p.t() @ h).to(_dt(c["dw"]))
    if op == "norm":
        t = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
        x = t.float()
        rr = (x.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = x * rr * s["gamma"]
        q, sc = _quantize(y) if c["out"] != "same" else (None, None)
        return (y.to(t.dtype) if c["out"] != "8bit" else None, None if s["r"] is None else t, q, sc, rr[:, 0])
    if op == "norm_grad":
        rr = s["rrms"][:, None]
        xh = s["x"].float() * rr
        dy = s["dy"].float()
        g = dy * s["gamma"]
        dx = rr * (g - xh * (g * xh).mean(1, keepdim=True))
        if s["ds"] is not None:
            dx = dx + s["ds"].float()
        return dx.to(s["x"].dtype), (dy * xh).sum(0)
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    live = [x if n is None else torch.where((torch.arange(x.shape[1], device="cuda") < n[:, None])[:, :, None], x,
                                            torch.zeros_like(x)) for x, n in zip(s["grads"], s["rows"])]
    for x in live:
        total += x.float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    factor = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    outs = [(x.float() * factor).to(x.dtype) for x in live]
    return torch.stack([norm.float(), factor]), outs


def _quantize(y):
    rows, d = y.shape
    yb = torch.nn.functional.pad(y, (0, -d % BLOCK)).reshape(rows, -1, BLOCK)
    top = yb.abs().amax(2).view(torch.int32)  # as bits: the exponent from bit 23 up, 448 = 1.75 * 2^8
    e = ((top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000)).clamp_min(127 + SCALE_MIN_EXP).to(torch.int32)
    q = (yb / (e << 23).view(torch.float32)[:, :, None]).to(torch.float8_e4m3fn)
    e = torch.nn.functional.pad(e, (0, -e.shape[1] % 4), value=127)
    return q.reshape(rows, -1)[:, :d].contiguous(), e.to(torch.uint8).view(torch.float8_e8m0fnu)


# ---------------------------------------------------------------- 64 bits


def _exact_8bit(y):
    """The values of y's e4m3 numbers and their scales, from 64-bit arithmetic."""
    rows, d = y.shape
    full = torch.zeros((rows, d + -d % BLOCK), dtype=torch.float64, device=y.device)
    full[:, :d] = y
    tiles = full.unfold(1, BLOCK, BLOCK)
    top = tiles.abs().max(-1).values
    sc = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=SCALE_MIN_EXP))
    sc = torch.where(top > E4M3_MAX * sc, 2 * sc, sc)  # where the logarithm was a last bit off
    sc = torch.where((top <= E4M3_MAX * sc / 2) & (sc > 2.0 ** SCALE_MIN_EXP), sc / 2, sc)
    v = tiles / sc[:, :, None]
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))  # e4m3: three bits behind the leading one
    step = torch.exp2(e - 3)
    v = (torch.round(v / step) * step).reshape(rows, -1)
    return v[:, :d], torch.nn.functional.pad(sc, (0, -sc.shape[1] % 4), value=1.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("loss", "loss_grad"):
        n, V = case["tokens"], case["vocab"]
        w, y = s["w"].double(), s["targets"].long()
        keep = torch.logical_and(y.ge(0), y.lt(V))
        first = torch.zeros((n,) if op == "loss" else (n, case["d"]), dtype=torch.float64, device="cuda")
        second = torch.zeros((n,) if op == "loss" else (V, case["d"]), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 27) // V)  # tokens at a time: 1 GB of logits
        for at in keep.nonzero()[:, 0].split(step):
            h = s["h"][at].double()
            x = torch.mm(h, w.t()).mul_(case["scale"])
            if op == "loss":
                lse = torch.logsumexp(x, 1)
                first[at], second[at] = lse - x[torch.arange(len(at), device="cuda"), y[at]], lse
                continue
            p = torch.exp_(x.sub_(s["lse"][at].double()[:, None]))
            p[torch.arange(len(at), device="cuda"), y[at]] -= 1.0
            p.mul_((s["dloss"][at].double() * case["scale"])[:, None])
            first[at] = torch.mm(p, w)
            second.addmm_(p.t(), h)
        return first, second
    if op == "norm":
        x = s["x"].double()
        if s["r"] is not None:  # rounded to the plan's type, as the residual stream holds it
            x = (x + s["r"].double()).to(s["x"].dtype).double()
        ms = (x * x).sum(1) / case["d"]
        rr = 1.0 / torch.sqrt(ms + EPS)
        y = x * (s["gamma"].double() * rr[:, None])
        q, sc = _exact_8bit(y) if case["out"] != "same" else (None, None)
        return (y if case["out"] != "8bit" else None), (None if s["r"] is None else x), q, sc, rr
    if op == "norm_grad":
        x, dy, rr = s["x"].double(), s["dy"].double(), s["rrms"].double()[:, None]
        x.mul_(rr)
        dgamma = torch.stack([(dy[i:i + 4096] * x[i:i + 4096]).sum(0) for i in range(0, len(dy), 4096)]).sum(0)
        dy.mul_(s["gamma"].double())
        inner = (dy * x).sum(1, keepdim=True) / case["d"]
        dx = dy.sub_(x.mul_(inner)).mul_(rr)
        if s["ds"] is not None:
            dx += s["ds"].double()
        return dx, dgamma
    squares, parts = [], []
    for x, n in zip(s["grads"], s["rows"]):
        x = x.double()
        if n is not None:
            for one, k in zip(x, n.tolist()):
                one[k:] = 0.0
        parts.append(x)
        squares.append(torch.dot(x.flatten(), x.flatten()))
    norm = torch.linalg.vector_norm(torch.stack(squares).sqrt())
    factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    for x in parts:
        x *= factor
    return torch.stack([norm, factor]), parts


def work(case):
    op, d = case["op"], case["d"]
    if op in ("loss", "loss_grad"):
        e, n, V = (2 if case["dtype"] == "bf16" else 4), case["tokens"], case["vocab"]
        reads = (n + V) * d * e + 4 * n
        if op == "loss":
            return dict(bytes=reads + 8 * n, flops=2 * n * V * d)
        return dict(bytes=reads + 8 * n + n * d * e + V * d * (2 if case["dw"] == "bf16" else 4), flops=6 * n * V * d)
    if op in ("norm", "norm_grad"):
        e, n = (2 if case["dtype"] == "bf16" else 4), case["rows"] * d
        if op == "norm_grad":
            return dict(bytes=(4 if case["residual"] else 3) * n * e + 8 * d + 4 * case["rows"], flops=8 * n)
        moved = n * e * (3 if case["residual"] else 1)
        moved += (n * e if case["out"] != "8bit" else 0) + (n + n // BLOCK if case["out"] != "same" else 0)
        return dict(bytes=moved + 4 * d + 4 * case["rows"], flops=6 * n)
    sizes = _clip_sizes(case)
    e = 2 if case["dtype"] == "bf16" else 4
    n = 0
    for i, k in enumerate(sizes):  # of the tables' rows half take part on average
        j = (i - 1) % 6 if i else -1
        n += k // 2 * 4 if j == 5 else k * (e if j < 1 else 4)
    return dict(bytes=2 * n + 8, flops=3 * sum(sizes))
