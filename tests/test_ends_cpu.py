"""Refusals of the operators at a model's ends, on the CPU: the library's own checks
(bad pointers never reach a launch) and the binding's."""

import ctypes as C
import math

import pytest
import torch

from test_operators_cpu import B, ODD, at, plan, refuses  # noqa: F401 (B is a fixture)


def off(p, n):
    return C.c_void_p(p.value + n)


def test_rms_norm_refusals(B):
    p = plan(B)
    fn = B.lib().engram_rms_norm
    rows, d = 33, 256
    bytes_ = rows * d * 2
    #       0     1      2      3     4      5     6      7      8      9      10     11
    good = [p._h, at(0), at(1), rows, at(2), 1e-6, at(3), at(4), at(5), at(6), at(7), None]
    refuses(fn, good, [(i, None) for i in (0, 1, 2, 4, 6, 8, 9)] + [(i, ODD) for i in (1, 2, 4, 6, 7, 8, 9, 10)] +
            [(3, 0), (3, -1), (5, -1.0), (5, math.nan), (5, math.inf),
             (6, off(at(0), 16)), (6, off(at(1), bytes_ - 16)), (6, at(2)), (7, at(2)), (7, off(at(0), 16)), (7, at(3)),
             (8, at(0)), (8, at(1)), (8, at(2)), (8, at(3)), (8, at(4)), (9, at(0)), (9, at(5)), (9, at(4)),
             (10, at(0)), (10, at(2)), (10, at(3)), (10, at(6)), (10, off(at(6), rows * 4 - 4))], B.E_INVALID_ARG)
    for bad in ([(7, None), (8, None), (9, None)],       # nothing is wanted
                [(2, off(at(0), 512)), (6, at(0))],      # in place of an input that the other lies across
                [(2, off(at(0), 512)), (7, at(0))], [(2, off(at(0), 512)), (7, off(at(0), 512))]):
        a = list(good)
        for i, v in bad:
            a[i] = v
        assert fn(*a) == B.E_INVALID_ARG, bad
    refuses(fn, good, [(3, 1 << 50)], B.E_UNSUPPORTED)
    wide = plan(B, d=32776)
    assert fn(wide._h, *good[1:]) == B.E_UNSUPPORTED
    assert wide.engram_rms_norm_backward_workspace_size(4) == 0


def test_rms_norm_backward_refusals(B):
    p = plan(B)
    ws = p.engram_rms_norm_backward_workspace_size(33)
    assert ws > 0 and p.engram_rms_norm_backward_workspace_size(0) == 0
    with pytest.raises(B.EngramError):
        p.rms_norm_backward_workspace(0)
    fn = B.lib().engram_rms_norm_backward
    #       0     1      2      3      4   5      6      7  8      9      10     11  12
    good = [p._h, at(0), at(1), at(2), 33, at(3), at(4), 0, at(5), at(6), at(7), ws, None]
    refuses(fn, good, [(i, None) for i in (0, 1, 2, 5, 6, 8, 9, 10)] + [(i, ODD) for i in (1, 2, 3, 5, 6, 8, 9)] +
            [(4, 0), (4, -7), (11, ws - 1), (10, off(at(7), 16)), (7, B.OUT_DELTA), (7, 1 << 20),
             (8, off(at(0), 16)), (8, off(at(1), 16)), (8, off(at(2), 16)), (8, at(3)), (8, at(4)), (9, at(0)), (9, at(2)),
             (9, at(3)), (9, at(5)), (10, at(0)), (10, at(2)), (10, at(5)), (10, at(6))], B.E_INVALID_ARG)
    refuses(fn, good, [(4, 1 << 50)], B.E_UNSUPPORTED)


def test_rms_norm_backward_workspace_serves_fewer_rows(B):
    for d in (8, 64, 256, 512, 2560, 2568, 4104, 8200, 16384, 32768):
        p = plan(B, d=d)
        sizes = [p.engram_rms_norm_backward_workspace_size(n) for n in sorted({2 ** i + j for i in range(21) for j in (0, 1, 3)})]
        assert sizes[0] > 0 and all(x <= y for x, y in zip(sizes, sizes[1:]))


def test_cross_entropy_refusals(B):
    p = plan(B)
    n = 33
    ws = p.engram_cross_entropy_workspace_size(n)
    assert ws > 0 and p.engram_cross_entropy_workspace_size(0) == 0 and p.engram_cross_entropy_workspace_size(-1) == 0
    with pytest.raises(B.EngramError):
        p.cross_entropy_workspace(0)
    fn = B.lib().engram_cross_entropy
    #       0     1      2      3      4  5    6      7      8      9   10
    good = [p._h, at(0), at(1), at(2), n, 1.0, at(3), at(4), at(5), ws, None]
    refuses(fn, good, [(i, None) for i in (0, 1, 2, 3, 6, 7, 8)] + [(i, ODD) for i in (1, 2, 3, 6, 7)] +
            [(4, 0), (4, -1), (5, math.nan), (5, -math.inf), (9, ws - 1), (8, off(at(5), 16)),
             (6, at(0)), (6, at(1)), (6, at(2)), (7, at(2)), (7, at(3)), (8, at(0)), (8, at(1)), (8, at(3)), (8, at(4)),
             (8, off(at(1), 1000 * 256 * 2 - 256))], B.E_INVALID_ARG)
    refuses(fn, good, [(4, (1 << 26) + 1), (4, 1 << 50)], B.E_UNSUPPORTED)
    for other in (plan(B, vocab=(1 << 22) + 1), plan(B, d=(1 << 20) + 8), plan(B, vocab=1 << 22, d=1 << 16)):
        assert fn(other._h, *good[1:]) == B.E_UNSUPPORTED
        assert other.engram_cross_entropy_workspace_size(n) == 0
        assert other.engram_cross_entropy_backward_workspace_size(n) == 0
    many = plan(B, vocab=1 << 22)  # 2^14 tiles wide: 2^8 rows of them
    assert many.engram_cross_entropy_workspace_size(255 * 256) > 0
    assert many.engram_cross_entropy_workspace_size(256 * 256) == 0


def test_cross_entropy_backward_refusals(B):
    p, f = plan(B), plan(B, dtype=B.F32)
    n = 33
    ws = p.engram_cross_entropy_backward_workspace_size(n)
    assert ws >= p.engram_cross_entropy_backward_workspace_size(n, torch.bfloat16) > 0
    assert f.engram_cross_entropy_backward_workspace_size(n, torch.bfloat16) == 0
    with pytest.raises(TypeError):
        p.engram_cross_entropy_backward_workspace_size(n, torch.float16)
    with pytest.raises(B.EngramError):
        f.cross_entropy_backward_workspace(n, torch.bfloat16)
    fn = B.lib().engram_cross_entropy_backward
    #       0     1      2      3      4  5    6      7      8    9  10     11     12     13     14  15
    good = [p._h, at(0), at(1), at(2), n, 1.0, at(3), at(4), 1.0, 0, at(5), at(6), B.F32, at(7), ws, None]
    refuses(fn, good, [(i, None) for i in (0, 1, 2, 3, 6, 13)] + [(i, ODD) for i in (1, 2, 3, 6, 7, 10, 11)] +
            [(4, 0), (4, -1), (5, math.nan), (8, math.inf), (9, B.OUT_DELTA), (9, 1 << 30), (12, 2), (12, -1),
             (14, ws - 1), (13, off(at(7), 16)), (10, at(0)), (10, at(1)), (10, at(2)), (10, at(3)), (10, at(4)),
             (11, at(0)), (11, at(1)), (11, at(4)), (11, at(5)), (13, at(0)), (13, at(1)), (13, at(5)), (13, at(6)),
             (11, off(at(1), 1000 * 256 * 2 - 16))], B.E_INVALID_ARG)
    a = list(good)
    a[10] = a[11] = None
    assert fn(*a) == B.E_INVALID_ARG  # nothing is wanted
    refuses(fn, good, [(4, (1 << 26) + 1)], B.E_UNSUPPORTED)
    a = list(good)
    a[0], a[12], a[14] = f._h, B.BF16, 1 << 40
    assert fn(*a) == B.E_UNSUPPORTED


@pytest.mark.parametrize("vocab,d", [(129280, 2560), (1000, 256), (50, 64), (1, 8), (200000, 1024), (17, 8192)])
def test_cross_entropy_workspaces_serve_smaller_batches(B, vocab, d):
    """The size never falls as the batch grows, across the thresholds of how the
    products are cut."""
    ns = sorted({max(1, 2 ** i + j) for i in range(18) for j in (-1, 0, 1, 7)} | set(range(1, 700, 13)) |
                {192 * 256 // (-(-vocab // 256)) + j for j in range(-300, 300, 37) if 192 * 256 // (-(-vocab // 256)) + j > 0})
    for dtype in (B.BF16, B.F32):
        p = plan(B, dtype=dtype, vocab=vocab, d=d)
        sizes = [[p.engram_cross_entropy_workspace_size(n) for n in ns],
                 [p.engram_cross_entropy_backward_workspace_size(n) for n in ns]]
        if dtype == B.BF16:
            sizes.append([p.engram_cross_entropy_backward_workspace_size(n, torch.bfloat16) for n in ns])
        for along in sizes:
            along = [s for s in along if s]
            assert len(along) > 40 and all(x <= y for x, y in zip(along, along[1:]))


def entry(B, data, n, out=None, counts=None, groups=1, rows=1, dtype=None):
    return B.GradC(data, out, counts, groups, rows, n, B.F32 if dtype is None else dtype)


def test_clip_grads_refusals(B):
    p = plan(B)
    fn = B.lib().engram_clip_grads
    ws = p.engram_clip_grads_workspace_size(3)
    assert ws > 0 and p.engram_clip_grads_workspace_size(0) == 0
    with pytest.raises(B.EngramError):
        p.clip_grads_workspace(0)

    def call(*es, n=None, max_norm=1.0, norm=at(20), w=at(21), size=ws, grads=True):
        arr = (B.GradC * max(1, len(es)))(*es)
        return fn(p._h, arr if grads else None, len(es) if n is None else n, max_norm, norm, w, size, None)

    def e(data, n, **kw):
        return entry(B, data, n, **kw)

    ok = e(at(0), 100, out=at(0))
    bad = [dict(n=0), dict(n=-1), dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(norm=None),
           dict(norm=ODD), dict(w=None), dict(w=off(at(21), 16)), dict(size=ws - 1), dict(grads=False), dict(norm=at(0)),
           dict(norm=at(21)), dict(w=off(at(0), -256)), dict(norm=off(at(0), 384))]
    for kw in bad:
        assert call(ok, **kw) == B.E_INVALID_ARG, kw
    for es in ([e(None, 5)], [e(ODD, 5)], [e(at(0), 5, out=ODD)], [e(at(0), -1)], [e(at(0), 5, groups=-1)],
               [e(at(0), 5, rows=-2)], [e(at(0), 5, dtype=2)], [e(at(0), 5, counts=off(at(3), 2))],
               [ok, e(at(0), 4)],                                # twice
               [ok, e(off(at(0), 384), 4)],                      # its last values
               [e(at(0), 100), e(at(1), 100, out=off(at(0), 16))],
               [e(at(0), 100, out=off(at(0), 16))],
               [e(at(0), 100, out=at(1)), e(at(2), 100, out=off(at(1), 384))],
               [e(at(0), 10, counts=at(1), groups=5, rows=4), e(at(1), 3)],
               [e(at(0), 10, counts=at(0), groups=5, rows=4)],
               [ok, e(at(5), 4, dtype=B.BF16), e(at(0), 4, dtype=B.BF16)]):
        assert call(*es) == B.E_INVALID_ARG, es
    for es in ([e(at(0), 1 << 43)], [e(at(0), 1 << 30, rows=1 << 30, groups=1 << 30)], [e(at(0), 1, groups=1 << 40)],
               [e(at(0), 1 << 41), e(at(30), 1 << 41), e(at(60), 1 << 41)]):
        assert call(*es) == B.E_UNSUPPORTED, es


def test_the_binding_refuses_tensors_of_another_kind(B):
    """Host tensors never reach the library."""
    p = plan(B)
    x, f, i32 = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros(256), torch.zeros(4, dtype=torch.int32)
    w, ws = torch.zeros((1000, 256), dtype=torch.bfloat16), torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: p.engram_rms_norm(x, f, x),
                 lambda: p.engram_rms_norm_backward(x, x, f, f[:4], x, f, ws),
                 lambda: p.engram_cross_entropy(x, w, i32, f[:4], f[:4], ws),
                 lambda: p.engram_cross_entropy_backward(x, w, i32, f[:4], None, x, w, ws),
                 lambda: B.GradList([f])):
        with pytest.raises(TypeError):
            call()


def test_the_binding_refuses_shapes(B, monkeypatch):
    def addr(t, name, *dtypes):
        if t is None:
            return None
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        if dtypes and t.dtype not in dtypes:
            raise TypeError(name)
        return t.data_ptr()

    monkeypatch.setattr(B, "_addr", addr)

    def never(*a):
        raise AssertionError("reached the launch")

    monkeypatch.setattr(B, "_call", never)
    p = plan(B)
    i32 = torch.zeros(4, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    f8 = lambda *s: torch.zeros(s).to(torch.float8_e4m3fn)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    ws, x, w, g = u8(1024), bf(4, 256), bf(1000, 256), f32(256)
    for call in (
            lambda: p.engram_rms_norm(bf(4, 248), g, bf(4, 248)),
            lambda: p.engram_rms_norm(x, f32(255), bf(4, 256)),
            lambda: p.engram_rms_norm(x, g, bf(5, 256)),
            lambda: p.engram_rms_norm(x, g, bf(4, 256), residual=bf(2, 256), total=bf(4, 256)),
            lambda: p.engram_rms_norm(x, g, bf(4, 256), residual=x, total=bf(2, 2, 256)),
            lambda: p.engram_rms_norm(x, g, q=f8(4, 248), scales=u8(4, 4)),
            lambda: p.engram_rms_norm(x, g, q=f8(4, 256), scales=u8(4, 2)),
            lambda: p.engram_rms_norm(x, g, q=f8(4, 256), scales=u8(1, 4)),
            lambda: p.engram_rms_norm(x, g, bf(4, 256), rrms=f32(3)),
            lambda: p.engram_rms_norm(bf(256, 4).t(), g, bf(4, 256)),
            lambda: p.engram_rms_norm_backward(x, bf(5, 256), g, f32(4), x, g, ws),
            lambda: p.engram_rms_norm_backward(x, x, g, f32(5), x, g, ws),
            lambda: p.engram_rms_norm_backward(x, x, g, f32(4), x, f32(4), ws),
            lambda: p.engram_rms_norm_backward(x, x, g, f32(4), x, g, ws, dtotal=bf(4, 4)),
            lambda: p.engram_cross_entropy(x, bf(999, 256), i32, f32(4), f32(4), ws),
            lambda: p.engram_cross_entropy(x, w, i32[:3], f32(4), f32(4), ws),
            lambda: p.engram_cross_entropy(x, w, i32, f32(5), f32(4), ws),
            lambda: p.engram_cross_entropy(x, w, i32, f32(4), f32(3), ws),
            lambda: p.engram_cross_entropy(bf(4, 128), w, i32, f32(4), f32(4), ws),
            lambda: p.engram_cross_entropy_backward(x, w, i32, f32(4), f32(3), x, f32(1000, 256), ws),
            lambda: p.engram_cross_entropy_backward(x, w, i32, f32(4), None, bf(5, 256), f32(1000, 256), ws),
            lambda: p.engram_cross_entropy_backward(x, w, i32, f32(4), None, x, f32(1001, 256), ws),
            lambda: p.engram_cross_entropy_backward(x, w, i32, f32(3), None, x, None, ws),
            lambda: B.GradList([]),
            lambda: B.GradList([f32(4)], outs=[f32(5)]),
            lambda: B.GradList([f32(4)], outs=[f32(4), f32(4)]),
            lambda: B.GradList([f32(4, 4).t()[:2]]),
            lambda: B.GradList([f32(4, 5)], row_counts=[i32[:3]]),
            lambda: B.GradList([f32(4)], row_counts=[i32])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: p.engram_rms_norm(x, bf(256), bf(4, 256)),
                 lambda: p.engram_rms_norm(x, g, f32(4, 256)),
                 lambda: p.engram_cross_entropy(x, w, i32.long(), f32(4), f32(4), ws),
                 lambda: p.engram_cross_entropy_backward(x, w, i32, f32(4), None, None, f32(1000, 256).half(), ws),
                 lambda: B.GradList([f32(4).half()]),
                 lambda: B.GradList([f32(4)], outs=[bf(4)]),
                 lambda: B.GradList([f32(4, 5)], row_counts=[i32.long()])):
        with pytest.raises(TypeError):
            call()


def test_a_gradient_list_of_several_shapes(B, monkeypatch):
    monkeypatch.setattr(B, "_addr", lambda t, name, *dtypes: None if t is None else t.data_ptr())
    g = [torch.zeros(5), torch.zeros((3, 4, 2, 7)), torch.zeros((0,)), torch.zeros((2, 6), dtype=torch.bfloat16)]
    counts = [None, torch.zeros(3, dtype=torch.int32), None, torch.zeros(2, dtype=torch.int32)]
    lst = B.GradList(g, row_counts=counts)
    assert [(e.n_groups, e.rows, e.row_len, e.dtype) for e in lst.c] == [
        (1, 1, 5, B.F32), (3, 4, 14, B.F32), (1, 1, 0, B.F32), (2, 6, 1, B.BF16)]
    assert all(e.out == e.data for e in lst.c)


def test_cross_entropy_refuses_scales_past_its_powers_of_two(B):
    """2^127 / ln 2 is the largest that fp32 holds: 2^127 passes, and what comes after it
    is refused; other arguments are bad, so that nothing is launched."""
    p = plan(B)
    ws, ws_b = p.engram_cross_entropy_workspace_size(33), p.engram_cross_entropy_backward_workspace_size(33)
    fwd, bwd = B.lib().engram_cross_entropy, B.lib().engram_cross_entropy_backward
    for sign in (1, -1):
        for scale, n, want in ((2.0 ** 127, 1 << 50, B.E_UNSUPPORTED), (2.0 ** 127 * (1 + 2.0 ** -23), 33, B.E_INVALID_ARG),
                               (3.4e38, 33, B.E_INVALID_ARG)):
            assert fwd(p._h, at(0), at(1), at(2), n, sign * scale, at(3), at(4), at(5), ws, None) == want
            assert bwd(p._h, at(0), at(1), at(2), n, sign * scale, at(3), at(4), 1.0, 0, at(5), at(6), B.F32, at(7), ws_b,
                       None) == want
