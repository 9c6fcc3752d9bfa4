"""Attention over the 4-bit cache with queries of every magnitude that bf16 holds.

Logits far past binary32's integers make the softmax one-hot: the row is the
value of its largest logit's token, whatever the logits' own rounding."""
import numpy as np
import pytest
import torch

import fp4_testlib as f4
from test_gpu_fp4 import OnGpu, bits, dev, kvq  # noqa: F401  (the fixture too)

pytestmark = pytest.mark.gpu

SCALES = [1e4, 1e6, 1e8, 1e10, 1e20, 1e30, 1e37, 3e37]


def widen(g, scales=SCALES):
    """Query head h of row j times scales[(h + 3 j) % n]."""
    q = f4.bf16_to_f32(g.q).astype(np.float64)
    j, h = np.arange(q.shape[0])[:, None], np.arange(q.shape[1])[None]
    q *= np.asarray(scales)[(h + 3 * j) % len(scales)][..., None]
    g.q = f4.to_bf16(q)
    g.dq = dev(g.q)


def check_one_hot(g, window=0, sinks=0):
    """Rows whose largest logit leads by more than its rounding are that token's value.

    A binary32 logit is off by at most 2^-18 S, S = sum |q_i K_i| / sqrt(dh) at its
    largest (fp4_testlib.attention), so a lead of 2^-16 S + 64 is at least 2^-17 S + 64
    in what the kernel sees, and the other weights are at most e^-64 each, e^-64 sum |V|
    together (0 as f16, but not where states of shared-out keys are merged).  Its own weight
    has an exponent of exactly 7, a power of two in f16, which the division takes out again:
    one binary32 rounding before the one to bf16."""
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0
    got = f4.bf16_to_f32(bits(g.out)).astype(np.float64)
    assert np.isfinite(got).all()
    b, K, V = g.b, f4.unit_values(g.K), f4.unit_values(g.V)
    G, seen_rows = b.hq // b.hkv, 0
    for s, L in enumerate(b.lens):
        n = int(g.cu[s + 1] - g.cu[s])
        t = np.arange(L)
        blk = b.table[s, t // 16]
        for j in range(n):
            pos = L - n + j
            ok = t <= pos
            if window:
                ok &= (t > pos - window) | (t < sinks)
            w = np.nonzero(ok)[0]
            for h in range(b.hkv):
                k = K[blk[w], h, w % 16] * float(b.ks[h % len(b.ks)])
                v = V[blk[w], h, w % 16] * float(b.vs[h % len(b.vs)])
                others = np.exp(-64.0) * np.abs(v).sum(0)
                q = f4.bf16_to_f32(g.q[g.cu[s] + j, h * G:(h + 1) * G]).astype(np.float64)
                x = q @ k.T / np.sqrt(b.dh)
                S = (np.abs(q) @ np.abs(k).T / np.sqrt(b.dh)).max(-1)
                for e in range(G):
                    top = np.sort(x[e])[-2:]
                    if len(top) == 2 and not top[1] - top[0] > 2.0 ** -16 * S[e] + 64:
                        continue
                    want = v[np.argmax(x[e])]
                    off = np.abs(got[g.cu[s] + j, h * G + e] - want)
                    bad = int((off > np.abs(want) * (2.0 ** -8 + 2.0 ** -20) + others).sum())
                    assert bad == 0, f"sequence {s} row {j} head {h * G + e}: {bad} values off"
                    seen_rows += 1
    assert seen_rows > 0.8 * got.shape[0] * b.hq


@pytest.mark.parametrize("lens,hq,hkv,dh", [
    ([300, 64, 5, 1], 8, 2, 128), ([300, 64, 5, 1], 8, 2, 64), ([5000], 32, 8, 128), ([1200, 3, 640, 77], 14, 2, 64),
    ([2300] * 20, 8, 8, 128), ([1700] * 24, 8, 8, 64), ([900, 2500, 17] * 6, 16, 4, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
def test_decode_large_logits(kvq, lens, hq, hkv, dh, window, sinks):  # noqa: F811
    b = f4.Batch(len(lens) + dh + window, lens, hq, hkv, dh)
    g = OnGpu(kvq, b, [1] * len(lens))
    widen(g)
    g.decode(window, sinks)
    check_one_hot(g, window, sinks)


@pytest.mark.parametrize("lens,counts,hq,hkv,dh", [
    ([300, 64, 5, 1], [40, 64, 5, 1], 8, 2, 128), ([300, 64, 5, 1], [30, 20, 1, 1], 8, 2, 64), ([2500], [3], 32, 8, 128),
    ([3001, 1700], [9, 4], 16, 4, 128), ([1000] * 6, [64, 7, 1, 30, 33, 16], 8, 2, 64), ([900, 20, 500], [70, 20, 40], 14, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
def test_prefill_large_logits(kvq, lens, counts, hq, hkv, dh, window, sinks):  # noqa: F811
    b = f4.Batch(sum(lens) + dh + window, lens, hq, hkv, dh)
    g = OnGpu(kvq, b, counts)
    widen(g)
    g.prefill(window, sinks)
    check_one_hot(g, window, sinks)


@pytest.mark.parametrize("dh", [64, 128])
def test_small_and_zero_queries(kvq, dh):  # noqa: F811
    """Queries down to bf16's subnormals, and of zero: the mean of the values, or nearly."""
    b = f4.Batch(5 + dh, [300, 64, 17], 8, 2, dh)
    for counts, call in (([1, 1, 1], "decode"), ([40, 64, 3], "prefill")):
        g = OnGpu(kvq, b, counts)
        widen(g, [1.0, 0.0, 1e-10, 1e-30, 1e-37, 3e-39, 30.0])
        getattr(g, call)()
        g.check(what=call)


@pytest.mark.parametrize("log2v", [-126, -118, 100])
@pytest.mark.parametrize("lens,counts,hq,hkv,dh", [
    ([300, 64, 17], [40, 64, 3], 8, 2, 64), ([2500], [3], 32, 8, 128), ([900] * 21, [5] * 21, 8, 8, 128),
    ([20000], [2], 8, 1, 64)])
def test_scales_near_the_ends(kvq, log2v, lens, counts, hq, hkv, dh):  # noqa: F811
    """Scales of V down to binary32's least normal one, and of K as far down with queries as
    far up.  Compared in units of V's scale, beside half of bf16's least step."""
    for n, call in (([1] * len(lens), "decode"), (counts, "prefill")):
        b = f4.Batch(len(lens) + dh, lens, hq, hkv, dh, per_head=False)
        g = OnGpu(kvq, b, n)
        b.vs = np.array([2.0 ** log2v], np.float32)
        if log2v < 0:
            g.q = f4.to_bf16(f4.bf16_to_f32(g.q) * np.float32(2.0 ** 111))  # (near-equal weights: large sums)
            b.ks = (b.ks * np.float32(2.0 ** -118)).astype(np.float32)
        g.ks, g.vs, g.dq = dev(b.ks), dev(b.vs), dev(g.q)
        getattr(g, call)()
        want, tol = f4.attention(g.q, g.K, g.V, b.ks, 1.0, b.table, b.lens, g.cu, 0, 0)
        torch.cuda.synchronize()
        assert int(g.st.item()) == 0
        off = np.abs(f4.bf16_to_f32(bits(g.out)).astype(np.float64) * 2.0 ** -log2v - want)
        bad = int((off > tol + 2.0 ** (-134 - log2v)).sum())
        assert bad == 0, f"{call}: {bad} of {off.size} values off, by up to {off.max():.3g}"


def test_decode_of_nothing(kvq):  # noqa: F811
    """Batches whose sequences are all empty, few of them and many."""
    for n, hkv in ((1, 1), (3, 2), (200, 8)):
        b = f4.Batch(n, [0] * n, 8, hkv, 128)
        g = OnGpu(kvq, b, [1] * n)
        g.decode()
        torch.cuda.synchronize()
        assert int(g.st.item()) == 0 and not bool(g.out.any())


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("lens,counts,hq,hkv", [([300, 150], [70, 40], 8, 2), ([2500], [4], 32, 8), ([700] * 20, [3] * 20, 8, 8)])
def test_bad_queries_stay_in_their_rows(kvq, dh, lens, counts, hq, hkv):  # noqa: F811
    """A NaN or an infinity in a query head is that head's output; its neighbours, which share
    matrix steps and decisions of a warp with it, are right."""
    for n, call in (([1] * len(lens), "decode"), (counts, "prefill")):
        b = f4.Batch(len(lens) + dh + 1, lens, hq, hkv, dh)
        g = OnGpu(kvq, b, n)
        q = f4.bf16_to_f32(g.q).copy()
        q[0, 0, 3], q[-1, hq - 1, dh - 1], q[-1, 1, 0] = np.nan, np.inf, -np.inf
        g.q = f4.to_bf16(q)
        g.dq = dev(g.q)
        getattr(g, call)()
        with np.errstate(invalid="ignore"):
            g.check(what=call)
        nan = torch.isnan(g.out.float())
        assert int(nan.any(-1).sum()) == 3 and bool(nan[0, 0].all())
