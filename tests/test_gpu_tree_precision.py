"""How far the tree attention's weights, scales and logits are from exact ones, where that shows."""
import math

import pytest
import torch

import step_testlib as lib
from step_testlib import E4M3, E5M2, PER_TENSOR, OnGpu, TreeBatch
from test_gpu_tree import kvq  # noqa: F401

pytestmark = pytest.mark.gpu


def fill(t, K, V, scale=1.0):
    """The batch's cache rows set to K and V [tokens][dh] (of one sequence and KV head), scales to `scale`."""
    for c, s, x in ((t.kc, t.ks, K), (t.vc, t.vs, V)):
        s.fill_(scale)
        at = torch.arange(x.shape[0], device="cuda")
        c.zero_()
        c[t.bt[0][at // 16].long(), 0, at % 16] = lib.encode(x.cuda() / scale, t.fmt)
    t.K, t.V = (lib.decode(c, t.fmt) * scale for c in (t.kc, t.vc))


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_weights_have_eleven_bits(kvq, fmt):  # noqa: F811
    """64 tokens whose weights lie at 1.12 to 1.17 of a power of two, where a step is largest next to them, against one
    that takes their sum away: what is left shows the weights' errors, not the output's rounding.

    The bound: half a step of bf16 of the output; for each weight half a step of its f16, 2^-11 (the values' magnitudes
    times weights), and 2^-24 of the row's largest (their magnitudes); 2^-18 for exp2, binary32 sums and logits (which
    are below 2^3, from queries that two E4M3 parts hold)."""
    n, dh = 256, 128
    t = TreeBatch([(65 + n, n)], 8, 1, dh, fmt, PER_TENSOR, kind="forest", seed=1)
    g = torch.Generator().manual_seed(2)
    K, V = torch.zeros(65 + n, dh), torch.zeros(65 + n, dh)
    K[1:65, 0], K[1:65, 1] = -16.0, -1.0
    V[0], V[1:65] = (-1.125 if fmt == E4M3 else -1.25), 1.0
    fill(t, K, V)
    q = torch.zeros(n, 8, dh)
    q[..., 0] = (4.0 + 0.04 * torch.rand(n, 8, generator=g)) * math.sqrt(dh) / 16
    q[..., 1] = 0.25 * torch.rand(n, 8, generator=g) + 0.02
    t.q = q.to(torch.bfloat16).cuda()
    x = t.q.double()[..., :2] @ torch.tensor([-16.0, -1.0], dtype=torch.float64, device="cuda") / math.sqrt(dh)
    a = torch.exp(x)  # (a node itself: a logit of 0, as the first token, and a value of 0)
    total = 2 + 64 * a
    v0 = float(V[0, 0])
    ref = (v0 + 64 * a) / total
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -18) * (abs(v0) + 64 * a) / total + 2.0 ** -24 * (abs(v0) + 64) / total
    o = OnGpu(kvq, t)
    o.call()
    torch.cuda.synchronize()
    assert int(o.st.item()) == 0
    err = (o.out.double() - ref[..., None]).abs()
    assert bool((err <= bound[..., None]).all()), float((err / bound[..., None]).max())
