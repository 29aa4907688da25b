"""The host side of the output head's cross entropy, run on the CPU: the tiles that
the library's own code chooses for a batch against the workspace that it lays out for
it (`tests/native/loss_cut_check.cpp`, compiled with the library's loss_cut.h)."""

import math
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hashed_gram_embedding_vocab_amd", "csrc")
F32, BF16 = 0, 1


def _hipcc():
    return os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def cuts(tmp_path_factory):
    """Of each (dtype, n_tok, vocab, d): tile, splits, cost, pieces, bytes written, bytes
    of the region, bytes of the workspace, costs of the gradients' products; None where the
    sizes are refused."""
    if not os.path.exists(_hipcc()):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("losscut") / "loss_cut_check")
    subprocess.check_call([_hipcc(), "-O2", "-std=c++17", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
                           os.path.join(ROOT, "tests", "native", "loss_cut_check.cpp"), os.path.join(CSRC, "loss_cut.cpp"),
                           "-o", exe])

    def ask(sizes):
        r = subprocess.run([exe], input="\n".join("%d %d %d %d" % s for s in sizes), capture_output=True, text=True,
                           timeout=120)
        assert r.returncode == 0, r.stderr
        lines = r.stdout.splitlines()
        assert len(lines) == len(sizes)
        return [None if l == "refused" else [float(x) if "." in x or "e" in x else int(x) for x in l.split()] for l in lines]

    return ask


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# heads whose weights pass a copy's piece, so that the logits are made in several
PIECED = [(F32, 190, 1453728, 12072), (F32, 111, 2869859, 16384), (BF16, 12288, 51698, 262088), (F32, 192, 40130, 6744),
          (BF16, 12502, 43767, 326240), (F32, 3234, 142127, 202360), (BF16, 12288, 4096, 1 << 20), (F32, 128, 65536, 8192)]


def test_sums_of_all_pieces_have_room(cuts):
    """Each piece of the vocabulary writes its tiles' maxima and sums behind those of the
    pieces before it."""
    rng = random.Random(1)
    sizes = list(PIECED)
    for _ in range(20000):
        dtype = rng.choice((F32, BF16))
        d = 8 * log_int(rng, 1, 1 << 17)
        sizes.append((dtype, log_int(rng, 65 if dtype == F32 else 12288, 1 << 17), log_int(rng, max(256, (1 << 27) // d), 1 << 22), d))
    seen = 0
    for s, a in zip(sizes, cuts(sizes)):
        if a is not None and a[3] > 1:
            seen += 1
            assert a[4] <= a[5], (s, a)
    assert seen > 4000


def test_every_cut_is_chosen_and_has_room(cuts):
    """Also where fp32 instructions run some tokens more than one tile's rows: the tile is
    one that the costs have, and the sums of it fit their region."""
    rng = random.Random(2)
    sizes = [(F32, n, 129280, d) for n in range(60, 90) for d in (8, 1024, 2560)]
    sizes += [(F32, 80, 1 << 22, 8), (F32, 373, 129280, 8), (BF16, 65, 129280, 2560), (F32, 65, 32833, 64)]
    sizes += [(rng.choice((F32, BF16)), log_int(rng, 1, 1 << 20), log_int(rng, 1, 1 << 22), 8 * log_int(rng, 1, 1 << 13))
              for _ in range(20000)]
    sizes += [(F32, log_int(rng, 60, 400), log_int(rng, 1 << 13, 1 << 22), 8 * log_int(rng, 1, 1 << 10)) for _ in range(5000)]
    seen = 0
    for s, a in zip(sizes, cuts(sizes)):
        if a is not None:
            seen += 1
            assert a[4] <= a[5], (s, a)
            assert max([a[2]] + a[7:]) < 1e20, (s, a)
    assert seen > 15000


def test_workspaces_of_more_tokens_are_no_smaller(cuts):
    """Across the thresholds of the forward's kinds of products, copies and pieces."""
    rng = random.Random(3)
    for _ in range(150):
        dtype, d = rng.choice((F32, BF16)), 8 * log_int(rng, 1, 1 << 15)
        vocab = log_int(rng, 1, 1 << 22)
        ns = sorted({log_int(rng, 1, 1 << 21) for _ in range(150)} | set(range(60, 130)))
        # (tokens up to which an fp32 plan multiplies by the fp32 instructions)
        direct = 80 + (300000000 // d + 350000) // vocab
        ns = sorted(set(ns) | {max(1, direct + j) for j in (-1, 0, 1, 2)})
        totals = [a[6] for a in cuts([(dtype, n, vocab, d) for n in ns]) if a is not None]
        assert all(x <= y for x, y in zip(totals, totals[1:])), (dtype, vocab, d)
