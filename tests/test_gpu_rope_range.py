"""kvq_rope_write's norm over all of bf16's range: a row's size cancels, whatever it is."""
import pytest
import torch

import step_testlib as lib
from step_testlib import BF16, BS, E4M3, E5M2, PER_HEAD, PER_TENSOR, PER_TOKEN_HEAD
from test_gpu_rope import Case, kvq  # noqa: F401

pytestmark = pytest.mark.gpu


def sized(c, low, high):
    """Each token's rows times a power of two of 2^low .. 2^high, neighbours far apart."""
    n = c.qkv.shape[0]
    e = torch.linspace(low, high, n, dtype=torch.float64)[torch.randperm(n, generator=torch.Generator().manual_seed(1))].round()
    x = c.qkv.double() * (2.0 ** e).cuda()[:, None]
    c.qkv.copy_(x.clamp(-3.3e38, 3.3e38).to(torch.bfloat16))


@pytest.mark.parametrize("fmt,gran,dh", [(E4M3, PER_HEAD, 128), (E5M2, PER_TOKEN_HEAD, 64), (BF16, PER_HEAD, 128), (E4M3, PER_TENSOR, 64)])
def test_rows_of_every_size(kvq, fmt, gran, dh):  # noqa: F811
    c = Case(kvq, 257, 6, 2, dh, fmt, gran, seed=21)
    sized(c, -20, 126)
    c.v.copy_(torch.randn(c.v.shape, generator=torch.Generator().manual_seed(2)))
    c.call()
    c.check()


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("low,high", [(-130, -60), (-130, 126)])
def test_rows_of_every_size_without_an_eps(kvq, dh, low, high):  # noqa: F811
    """An eps of 0: rows down to the subnormals are normed as others are.  Same bound as with one: 2^-8 of the output, 2^-18
    of its pair."""
    c = Case(kvq, 200, 5, 3, dh, BF16, seed=22, skip=False)
    sized(c, low, high)
    ordinary = (c.q.double().abs().amax(-1) > 0) & (c.k.double().abs().amax(-1).amin(-1, keepdim=True) > 0)
    assert bool(ordinary.all())
    c.call(eps=0.0)
    torch.cuda.synchronize()
    for x, w, got in ((c.q, c.wq, c.out), (c.k, c.wk, c.caches[0][c.slots // BS, :, c.slots % BS])):
        z, size = lib.rotated(x, w, 0.0, c.pos, c.freq, c.axis, c.inter)
        assert bool(((got.double() - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -18 * size).all())


def test_rows_beside_ones_that_are_not_finite(kvq):  # noqa: F811
    """A NaN, an infinity and rows of zeros among rows of every size: the others keep their bits."""
    a, b = (Case(kvq, 64, 8, 4, 128, E4M3, seed=23, skip=False) for _ in range(2))
    for c in (a, b):
        sized(c, -20, 126)
    b.q[3, 2, 5], b.q[9, 0, 0], b.k[20, 1, 7] = float("nan"), float("inf"), -float("inf")
    b.q[11, 4], b.k[30, 2] = 0.0, 0.0
    for c in (a, b):
        c.call()
    torch.cuda.synchronize()
    keep_q, keep_k = torch.ones(64, 8, dtype=torch.bool, device="cuda"), torch.ones(64, 4, dtype=torch.bool, device="cuda")
    for row in ((3, 2), (9, 0), (11, 4)):
        keep_q[row] = False
    for row in ((20, 1), (30, 2)):
        keep_k[row] = False
    assert torch.equal(a.out[keep_q], b.out[keep_q]) and bool((b.out[11, 4] == 0).all())
    got, want = (x.caches[0][x.slots // BS, :, x.slots % BS] for x in (b, a))
    assert torch.equal(got[keep_k], want[keep_k]) and bool((got[30, 2] & 0x7F == 0).all())
    assert bool(b.out[3, 2].isnan().all())
