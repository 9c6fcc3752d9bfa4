"""Trees of few blocks, several to a CTA: what a piece's warps hand each other is theirs, however late one of them is.

The test build has a hook that puts one softmax warp to sleep for 20 us before it reads the logits' scales of a piece and
before it looks whether NaN have to be put back; all waits stay as they are."""
import ctypes

import pytest
import torch

import step_testlib as lib
from step_testlib import BF16, E4M3, E5M2, PER_HEAD, PER_TOKEN_HEAD
from test_gpu_step_wait_timeout import call, hooked  # noqa: F401
from test_gpu_tree import kvq  # noqa: F401
from test_gpu_tree_precision import check_scaled
from test_gpu_wait_timeout import tlib  # noqa: F401

pytestmark = pytest.mark.gpu


def batch(fmt, gran, dh, B=320, kind="tree"):
    """Some five pieces a CTA, of one to three blocks and up to 128 rows; queries of another size in each sequence."""
    g = torch.Generator().manual_seed(dh + fmt)
    seqs = [(n + int(torch.randint(1, 180, (1,), generator=g)), n) for n in (int(torch.randint(9, 17, (1,), generator=g)) for _ in range(B))]
    b = lib.TreeBatch(seqs, 16, 2, dh, fmt, gran, kind=kind, seed=fmt)
    size = torch.repeat_interleave(2.0 ** torch.randint(-6, 3, (B,), generator=g), torch.tensor(b.nodes)).to(torch.bfloat16)
    b.q *= size.cuda()[:, None, None]
    return b


def with_nan(b):
    """NaN in a value of a node of every third sequence: the rows (and dims) that see it."""
    where = torch.zeros(b.q.shape, dtype=torch.bool, device="cuda")
    for i in range(0, len(b.lens), 3):
        L, n = b.lens[i], b.nodes[i]
        node, head, d = (5 * i) % n, i % b.hkv, (7 * i) % b.dh
        t = L - n + node
        b.vc[int(b.bt[i, t // 16]), head, t % 16, d] = float("nan") if b.fmt == BF16 else 0x7F
        G = b.hq // b.hkv
        for j in range(n):
            if node in lib.way_up(b.parents[i], j):
                where[int(b.cu[i]) + j, head * G:(head + 1) * G, d] = True
    return where


CASES = [(E4M3, PER_HEAD, 128), (BF16, PER_HEAD, 128), (E4M3, PER_TOKEN_HEAD, 64), (E5M2, PER_HEAD, 64)]


@pytest.mark.parametrize("fmt,gran,dh", CASES)
def test_short_pieces(kvq, hooked, fmt, gran, dh):  # noqa: F811
    b = batch(fmt, gran, dh)
    g = lib.OnGpu(kvq, b)
    g.call()
    check_scaled(g) if gran == PER_TOKEN_HEAD else g.check()
    clean = g.out.clone()
    where = with_nan(b)
    hooked.kvq_test_late_warp.restype, hooked.kvq_test_late_warp.argtypes = None, [ctypes.c_int]

    def same(what):
        torch.cuda.synchronize()
        assert int(g.st.item()) == 0, what
        assert torch.equal(g.out.isnan(), where), what
        assert torch.equal(g.out[~where], clean[~where]), what

    for i in range(5):
        g.out.fill_(7.0)
        g.call()
        same(f"run {i}")
    try:
        for warp in range(12):
            hooked.kvq_test_late_warp(warp)
            g.out.fill_(7.0)
            call(hooked, g)
            same(f"warp {warp} late")
    finally:
        hooked.kvq_test_late_warp(-1)


@pytest.mark.parametrize("kind", ["chain", "star"])
def test_short_pieces_of_chains_and_stars(kvq, kind):  # noqa: F811
    """Walks up of very different lengths before the scales are read."""
    b = batch(E4M3, PER_HEAD, 128, kind=kind)
    g = lib.OnGpu(kvq, b)
    g.call()
    g.check()
    clean = g.out.clone()
    where = with_nan(b)
    for _ in range(5):
        g.out.fill_(7.0)
        g.call()
        torch.cuda.synchronize()
        assert torch.equal(g.out.isnan(), where) and torch.equal(g.out[~where], clean[~where])
