"""Refusals of the operators beside the layer, on the CPU: the library's own
checks (bad pointers never reach a launch) and the binding's."""

import ctypes as C
import math
import os

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from hashed_gram_embedding_vocab_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from hashed_gram_embedding_vocab_amd import build
        build.build()
    binding.lib()
    if torch.cuda.is_available():
        pytest.skip("fake-pointer validation tests run only where no GPU exists")
    return binding


def plan(B, dtype=None, d=256, vocab=1000, n_branches=2):
    return B.Plan(vocab=vocab, vocab_comp=770, heads=4, head_dim=32, table_rows=[10007] * 8, hash_seed=1, d_model=d,
                  n_branches=n_branches, dtype=B.BF16 if dtype is None else dtype)


def at(n):
    """The n-th of well separated fake buffers."""
    return C.c_void_p((n + 1) << 40)


ODD = C.c_void_p((77 << 40) + 4)


def refuses(fn, good, bad, status):
    for i, v in bad:
        a = list(good)
        a[i] = v
        assert fn(*a) == status, (i, v)


def test_embed_refusals(B):
    p = plan(B)
    fn = B.lib().engram_embed
    good = [p._h, at(0), 33, at(1), 1.0, at(2), None, None]
    table_bytes, h_bytes = 1000 * 256 * 2, 2 * 33 * 256 * 2
    refuses(fn, good, [(0, None), (1, None), (3, None), (5, None), (2, 0), (2, -1), (1, ODD), (3, ODD), (5, ODD),
                       (4, math.nan), (4, math.inf),
                       (5, at(1)), (5, C.c_void_p(at(1).value + table_bytes - 16)),
                       (5, C.c_void_p(at(1).value - h_bytes + 16)), (5, at(0)), (6, at(0)), (6, at(1)), (6, at(2)),
                       (6, C.c_void_p(at(2).value + h_bytes - 4)), (6, C.c_void_p(at(7).value + 2))], B.E_INVALID_ARG)
    refuses(fn, good, [(2, 1 << 31)], B.E_UNSUPPORTED)
    wide = plan(B, d=1 << 24, vocab=1 << 20)
    assert fn(wide._h, *good[1:]) == B.E_UNSUPPORTED


def test_embed_backward_refusals(B):
    p = plan(B)
    n = 100
    ws = p.engram_embed_backward_workspace_size(n)
    # order, ids, starts and two fp32 parts of every 32 positions
    assert ws >= 8 * n + 4 * 1001 + 2 * 4 * 256 * 4
    assert p.engram_embed_backward_workspace_size(0) == 0
    assert p.engram_embed_backward_workspace_size(-3) == 0
    assert p.engram_embed_backward_workspace_size(1 << 31) == 0
    with pytest.raises(B.EngramError):
        p.embed_backward_workspace(0)
    fn = B.lib().engram_embed_backward
    good = [p._h, at(0), n, at(1), 1.0, 0, at(2), at(3), ws, None]
    refuses(fn, good, [(0, None), (1, None), (3, None), (6, None), (7, None), (2, 0), (2, -5), (1, ODD), (3, ODD),
                       (6, ODD), (7, C.c_void_p(at(3).value + 16)), (8, ws - 1), (4, math.nan), (4, -math.inf),
                       (5, B.OUT_DELTA), (5, B.QUANTIZE_TRANSPOSE), (5, 1 << 30),
                       (6, at(1)), (6, at(0)), (7, at(2)), (7, at(1)), (7, at(0))], B.E_INVALID_ARG)
    refuses(fn, good, [(2, 1 << 31)], B.E_UNSUPPORTED)
    assert plan(B, vocab=(1 << 31) - 1).engram_embed_backward_workspace_size(4) == 0
    assert plan(B, vocab=1 << 20, d=1 << 24).engram_embed_backward_workspace_size(4) == 0
    assert plan(B, vocab=8, d=1 << 26).engram_embed_backward_workspace_size(512) == 0


def test_layer_norm_refusals(B):
    p = plan(B)
    fn = B.lib().engram_layer_norm
    good = [p._h, at(0), 33, at(1), at(2), 1e-5, at(3), at(4), at(5), None]
    refuses(fn, good, [(0, None), (1, None), (3, None), (6, None), (2, 0), (2, -1), (1, ODD), (3, ODD), (4, ODD),
                       (6, ODD), (7, ODD), (8, ODD), (5, -1.0), (5, math.nan), (5, math.inf),
                       (6, C.c_void_p(at(0).value + 16)), (6, at(1)), (6, at(2)), (7, at(0)), (8, at(0)), (7, at(3)),
                       (8, at(3)), (8, at(4)), (7, at(1)), (8, at(2))], B.E_INVALID_ARG)
    refuses(fn, good, [(2, 1 << 50)], B.E_UNSUPPORTED)
    wide = plan(B, d=32776)
    assert fn(wide._h, *good[1:]) == B.E_UNSUPPORTED
    assert wide.engram_layer_norm_backward_workspace_size(4) == 0


def test_layer_norm_backward_refusals(B):
    p = plan(B)
    ws = p.engram_layer_norm_backward_workspace_size(33)
    assert ws > 0 and p.engram_layer_norm_backward_workspace_size(0) == 0
    with pytest.raises(B.EngramError):
        p.layer_norm_backward_workspace(0)
    fn = B.lib().engram_layer_norm_backward
    #        0     1      2      3   4      5      6      7  8      9      10     11     12  13
    good = [p._h, at(0), at(1), 33, at(2), at(3), at(4), 0, at(5), at(6), at(7), at(8), ws, None]
    refuses(fn, good, [(i, None) for i in (0, 1, 2, 4, 5, 6, 8, 9, 11)] + [(i, ODD) for i in (1, 2, 4, 5, 6, 8, 9, 10)] +
            [(3, 0), (3, -1), (12, ws - 1), (11, C.c_void_p(at(8).value + 16)), (7, B.OUT_DELTA), (7, 1 << 20),
             (8, C.c_void_p(at(0).value + 16)), (8, C.c_void_p(at(1).value + 16)), (8, at(2)), (8, at(3)), (8, at(4)),
             (9, at(0)), (9, at(2)), (9, at(5)), (10, at(6)), (10, at(1)), (11, at(0)), (11, at(5)), (11, at(7))],
            B.E_INVALID_ARG)


def test_quantize_refusals(B):
    p = plan(B)
    fn = B.lib().engram_quantize_fp8
    good = [p._h, at(0), 33, 256, 1, 0, at(1), at(2), None]
    refuses(fn, good, [(0, None), (1, None), (6, None), (7, None), (2, 0), (2, -1), (3, 0), (3, -128), (4, 0), (4, 2),
                       (4, 64), (4, -1), (5, B.GRAD_ACCUMULATE), (5, 1), (1, ODD), (6, ODD), (7, ODD), (6, at(0)),
                       (7, at(0)), (7, at(1)), (6, C.c_void_p(at(0).value + 33 * 256 * 2 - 16))], B.E_INVALID_ARG)
    refuses(fn, good, [(2, 1 << 50), (2, 1 << 31), (3, 1 << 31)], B.E_UNSUPPORTED)


def test_matmul_refusals(B):
    p = plan(B)
    fn = B.lib().engram_matmul_fp8
    for m, n, k in [(33, 100, 256), (256, 256, 1 << 17)]:
        ws = p.engram_matmul_fp8_workspace_size(m, n, k)
        #        0     1      2     3   4      5      6   7  8  9  10     11     12     13  14
        good = [p._h, at(0), at(1), 1, at(2), at(3), 128, m, n, k, at(4), B.F32, at(5), ws, None]
        bad = [(i, None) for i in (0, 1, 2, 4, 5, 10)] + [(i, ODD) for i in (1, 2, 4, 5, 10)] + [
            (3, 0), (3, 16), (6, 2), (6, -128), (7, 0), (8, 0), (9, 0), (7, -1), (8, -1), (9, -16), (11, 2), (11, -1),
            (10, at(0)), (10, at(1)), (10, at(2)), (10, at(3))]
        if ws:
            bad += [(12, None), (12, C.c_void_p(at(5).value + 16)), (13, ws - 1)] + [(12, at(i)) for i in range(5)]
        refuses(fn, good, bad, B.E_INVALID_ARG)
        refuses(fn, good, [(9, 24), (9, 250), (9, 1 << 22), (7, 1 << 45), (8, 1 << 45)], B.E_UNSUPPORTED)
    assert p.engram_matmul_fp8_workspace_size(5, 5, 24) == 0
    assert p.engram_matmul_fp8_workspace_size(0, 5, 32) == 0
    assert p.matmul_fp8_workspace(0, 5, 32, device="cpu") is None


def test_the_binding_refuses_tensors_of_another_kind(B):
    """Host tensors never reach the library."""
    p = plan(B)
    i32, bf = torch.zeros(4, dtype=torch.int32), torch.zeros((1000, 256), dtype=torch.bfloat16)
    x, f = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros(256)
    q, s = torch.zeros((4, 256)).to(torch.float8_e4m3fn), torch.zeros((4, 4), dtype=torch.uint8)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: p.engram_embed(i32, bf, torch.zeros((2, 4, 256), dtype=torch.bfloat16)),
                 lambda: p.engram_embed_backward(i32, torch.zeros((2, 4, 256), dtype=torch.bfloat16),
                                                 torch.zeros((1000, 256)), ws),
                 lambda: p.engram_layer_norm(x, f, None, x),
                 lambda: p.engram_layer_norm_backward(x, x, f, f[:4], f[:4], x, f, None, ws),
                 lambda: p.engram_quantize_fp8(x, q, s),
                 lambda: p.engram_matmul_fp8(q, s, q, s, torch.zeros((4, 4)))):
        with pytest.raises(TypeError):
            call()



def test_the_binding_refuses_shapes(B, monkeypatch):
    """Shapes, types and contiguity are checked before the library is called (the
    tensors stand on the CPU here, with the device check taken out of the way)."""
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
    ws = u8(1024)
    for call in (
            lambda: p.engram_embed(i32, bf(999, 256), bf(2, 4, 256)),
            lambda: p.engram_embed(i32, bf(1000, 256), bf(1, 4, 256)),
            lambda: p.engram_embed(i32, bf(1000, 256), bf(2, 5, 256)),
            lambda: p.engram_embed(i32, bf(1000, 256), bf(2, 4, 256), bad_tokens=i32[:0]),
            lambda: p.engram_embed(torch.zeros(8, dtype=torch.int32)[::2], bf(1000, 256), bf(2, 4, 256)),
            lambda: p.engram_embed_backward(i32, bf(2, 3, 256), f32(1000, 256), ws),
            lambda: p.engram_embed_backward(i32, bf(2, 4, 256), f32(1001, 256), ws),
            lambda: p.engram_layer_norm(bf(4, 248), f32(256), None, bf(4, 248)),
            lambda: p.engram_layer_norm(bf(4, 256), f32(248), None, bf(4, 256)),
            lambda: p.engram_layer_norm(bf(4, 256), f32(256), f32(255), bf(4, 256)),
            lambda: p.engram_layer_norm(bf(4, 256), f32(256), None, bf(3, 256)),
            lambda: p.engram_layer_norm(bf(4, 256), f32(256), None, bf(4, 256), mean=f32(3)),
            lambda: p.engram_layer_norm(bf(4, 256), f32(256), None, bf(4, 256), rstd=f32(5)),
            lambda: p.engram_layer_norm(bf(256, 4).t(), f32(256), None, bf(4, 256)),
            lambda: p.engram_layer_norm_backward(bf(4, 256), bf(4, 256), f32(256), f32(4), f32(4), bf(4, 256),
                                                 f32(255), None, ws),
            lambda: p.engram_layer_norm_backward(bf(4, 256), bf(5, 256), f32(256), f32(4), f32(4), bf(4, 256),
                                                 f32(256), None, ws),
            lambda: p.engram_layer_norm_backward(bf(4, 256), bf(4, 256), f32(256), f32(4), f32(1), bf(4, 256),
                                                 f32(256), None, ws),
            lambda: p.engram_quantize_fp8(bf(4, 256), f8(256, 4), u8(4, 4)),
            lambda: p.engram_quantize_fp8(bf(4, 256), f8(4, 256), u8(4, 2)),
            lambda: p.engram_quantize_fp8(bf(4, 256), f8(4, 256), u8(4, 4), block_rows=128),
            lambda: p.engram_quantize_fp8(bf(2, 2, 256), f8(4, 256), u8(4, 4)),
            lambda: p.engram_matmul_fp8(f8(4, 256), u8(4, 4), f8(5, 240), u8(1, 4), f32(4, 5)),
            lambda: p.engram_matmul_fp8(f8(4, 256), u8(4, 4), f8(5, 256), u8(5, 4), f32(4, 5)),
            lambda: p.engram_matmul_fp8(f8(4, 256), u8(4, 4), f8(5, 256), u8(1, 4), f32(5, 4)),
            lambda: p.engram_matmul_fp8(f8(4, 256), u8(1, 4), f8(5, 256), u8(1, 4), f32(4, 5))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: p.engram_embed(i32.long(), bf(1000, 256), bf(2, 4, 256)),
                 lambda: p.engram_embed(i32, f32(1000, 256), bf(2, 4, 256)),
                 lambda: p.engram_layer_norm(bf(4, 256), bf(256), None, bf(4, 256)),
                 lambda: p.engram_matmul_fp8(f8(4, 256), u8(4, 4), f8(5, 256), u8(1, 4), torch.zeros(4, 5).half())):
        with pytest.raises(TypeError):
            call()


def test_one_device_and_its_stream(B, monkeypatch):
    """Tensors on two devices, or a stream of another device, are refused; the
    tensors' device is the current one during the call, on its current stream."""
    class T:
        def __init__(self, d):
            self.d = d

        def get_device(self):
            return self.d

    class S:
        cuda_stream = 5

        def __init__(self, d):
            self.device = torch.device("cuda", d)

    seen = []

    class Guard:
        def __init__(self, d):
            seen.append("device %d" % d)

        def __enter__(self):
            return self

        def __exit__(self, *a):
            seen.append("left")

    class Lib:
        @staticmethod
        def engram_thing(*a):
            seen.append(a)
            return B.E_UNSUPPORTED if a[0] == "bad" else B.OK

        engram_status_string = staticmethod(lambda s: b"said so")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(B, "_current_raw_stream", lambda d: 70 + d)
    monkeypatch.setattr(B, "lib", lambda: Lib)
    with pytest.raises(ValueError):
        B._call("engram_thing", None, (T(0), None, T(1)), 1)
    with pytest.raises(ValueError):
        B._call("engram_thing", S(1), (T(0),), 1)
    assert seen == []
    B._call("engram_thing", S(0), (T(0), None), 1, 2)
    B._call("engram_thing", None, (T(0), T(0)), 3)
    assert seen == [(1, 2, 5), (3, 70)]
    B._call("engram_thing", None, (T(1), T(1)), 4)
    B._call("engram_thing", S(1), (T(1),), 5)
    assert seen[2:] == ["device 1", (4, 71), "left", "device 1", (5, 5), "left"]
    with pytest.raises(B.EngramError):
        B._call("engram_thing", None, (T(0),), "bad")


def test_scale_shape(B):
    for cols, pitch in ((1, 4), (128, 4), (129, 4), (512, 4), (513, 8), (1280, 12), (16384, 128)):
        assert B.Plan.fp8_scale_shape(300, cols, 1) == (300, pitch)
        assert B.Plan.fp8_scale_shape(300, cols, 128) == (3, pitch)


@pytest.mark.parametrize("vocab,d", [(129280, 2560), (1000, 8), (1000, 512), (50, 520), (700, 1 << 14), (9, 1 << 23)])
def test_an_embed_backward_workspace_serves_smaller_batches(B, vocab, d):
    """The size never falls as the batch grows, also where its chunks become longer."""
    p = plan(B, vocab=vocab, d=d, n_branches=1)
    turn = 65536 // ((d + 511) // 512)  # from here on a chunk is 32 tokens
    ns = {1, 2, 7, 8, 9, 100, 512, 513, 1000, 2 * turn, 3 * turn, 4 * turn + 5, 5 * turn, 1 << 20}
    ns |= {turn + i for i in range(-40, 41)} | {turn * i // 16 for i in range(1, 80)}
    sizes = [s for n in sorted(ns) if n > 0 for s in [p.engram_embed_backward_workspace_size(n)] if s]
    assert len(sizes) > 10
    assert all(x <= y for x, y in zip(sizes, sizes[1:]))
    # and is enough for two rows a chunk of this batch
    for n in sorted(ns):
        s = p.engram_embed_backward_workspace_size(n) if n > 0 else 0
        if s:
            chunk = 32 if n * ((d + 511) // 512) >= 65536 else 8
            assert s >= 8 * n + 4 * (vocab + 1) + 8 * d * -(-n // chunk)


def test_a_matmul_workspace_serves_smaller_products(B):
    """The size never falls as a batch grows, be it the product's rows (a
    projection) or its contraction (a weight gradient), across the thresholds of
    how a product is cut, and no larger size is refused its own."""
    p = plan(B)
    size = p.engram_matmul_fp8_workspace_size
    steps = sorted({max(1, 2 ** i + j) for i in range(17) for j in (-1, 0, 1, 5)} | {2560, 1280, 4096, 12800, 129280})
    ks = sorted({16 * max(1, s // 16) for s in steps} | {16 * s for s in (160, 161, 176, 255, 1024, 2047, 2048, 131072)})
    fixed = [(1, 16), (16, 8192), (16, 8193), (17, 128), (100, 129), (129, 2560), (1280, 2560), (2560, 2560), (4096, 12800)]
    for a, b in fixed:
        for kk in (128, 1280, 2048, 2560, 8192, 32768, 1 << 20):
            for along in ([size(m, a, kk) for m in steps], [size(b, n, kk) for n in steps], [size(a, n, kk) for n in steps]):
                assert all(x <= y for x, y in zip(along, along[1:]))
        along = [size(a, b, k) for k in ks]
        assert all(x <= y for x, y in zip(along, along[1:]))
    assert max(size(m, n, 4194288) for m in steps for n in steps) <= 64 << 20
    # parts of K that a shape used before its size covered smaller ones
    assert size(4096, 2560, 2560) >= 52428800      # 2560 rows in two parts
    assert size(4096, 1280, 32768) >= 5 * 2560 * 1280 * 4
    assert size(2560, 1280, 32768) >= 5 * 2560 * 1280 * 4


def test_matmul_sizes_up_to_the_launchs(B):
    """What is refused as unsupported is what one launch's tiles do not cover: a
    misaligned result is found behind that check, and nothing is launched."""
    p = plan(B)
    fn = B.lib().engram_matmul_fp8
    call = lambda m, n, k: fn(p._h, at(0), at(1), 1, at(2), at(3), 1, m, n, k, ODD, B.BF16, None, 0, None)  # noqa: E731
    for m, n, k in [(131072, 262144, 128), (1048576, 32768, 1280), (1 << 20, 1 << 18, 16), (100, (1 << 31) - 128, 16),
                    ((1 << 31) - 128, 1, 16), ((1 << 23) * 256 - 256, 256, 16)]:
        assert call(m, n, k) == B.E_INVALID_ARG, (m, n, k)
    for m, n, k in [(100, 1 << 31, 16), (1 << 31, 1, 16), ((1 << 23) * 256, 129, 16)]:
        assert call(m, n, k) == B.E_UNSUPPORTED, (m, n, k)


def test_a_layer_norm_backward_workspace_serves_fewer_rows(B):
    for d in (8, 64, 256, 512, 2560, 2568, 4104, 8200, 16384, 32768):
        p = plan(B, d=d)
        sizes = [p.engram_layer_norm_backward_workspace_size(n) for n in sorted({2 ** i + j for i in range(21) for j in (0, 1, 3)})]
        assert sizes[0] > 0 and all(x <= y for x, y in zip(sizes, sizes[1:]))
