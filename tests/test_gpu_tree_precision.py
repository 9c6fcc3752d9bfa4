"""How far the tree attention's weights, scales and logits are from exact ones, where that shows."""
import math

import pytest
import torch

import step_testlib as lib
from step_testlib import BF16, E4M3, E5M2, PER_HEAD, PER_TENSOR, PER_TOKEN_HEAD, OnGpu, TreeBatch
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


@pytest.mark.parametrize("fmt,dh", [(E4M3, 128), (E5M2, 128), (E4M3, 64)])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("outlier", [2.0 ** 30, 2.0 ** 100, math.inf, math.nan])
def test_scales_of_tokens_that_a_row_does_not_see(kvq, fmt, dh, window, outlier):  # noqa: F811
    """Outliers among the scales, K's and V's, of two nodes and of tokens about the window's start: the rows that do not
    see them keep their bits, those that see a NaN are NaN."""
    b = TreeBatch([(300, 30), (90, 20), (2000, 16)], 8, 2, dh, fmt, PER_TOKEN_HEAD, window=window, seed=31)
    clean = OnGpu(kvq, b)
    clean.call()
    clean.check()
    P = 270
    nodes, before = (4, 11), ((P - 33, P - 60) if window else ())
    for i, t in enumerate([P + j for j in nodes] + list(before)):
        for s in (b.ks, b.vs) if i % 2 else (b.vs,):
            s[int(b.bt[0, t // 16]), 1, t % 16] = outlier
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0
    assert torch.equal(g.out[:, :4], clean.out[:, :4]) and torch.equal(g.out[30:], clean.out[30:])
    saw = 0
    for j in range(30):
        way = lib.way_up(b.parents[0], j)
        near = way[:window] if window else way
        first = max(0, P + len(way) - window) if window else 0
        sees = any(n in near for n in nodes) or any(t >= first for t in before)
        saw += sees
        if not sees:
            assert torch.equal(g.out[j, 4:], clean.out[j, 4:]), j
        elif math.isnan(outlier):
            assert bool(g.out[j, 4:].isnan().all()), j
    assert saw >= 2  # (a window of 40 shows every node the token 33 before the tree)


@pytest.mark.parametrize("outlier", [2.0 ** 30, math.inf, math.nan])
def test_scales_before_the_window(kvq, outlier):  # noqa: F811
    """A chain of drafts: outliers among the scales of tokens that leave the window one node after the other."""
    window, P = 40, 270
    b = TreeBatch([(300, 30), (2000, 16)], 8, 2, 128, E4M3, PER_TOKEN_HEAD, window=window, kind="chain", seed=33)
    clean = OnGpu(kvq, b)
    clean.call()
    clean.check()
    before = (P - 33, P - 30, P - 60)
    for i, t in enumerate(before):
        for s in (b.ks, b.vs) if i == 1 else (b.vs,):
            s[int(b.bt[0, t // 16]), 1, t % 16] = outlier
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    assert torch.equal(g.out[:, :4], clean.out[:, :4]) and torch.equal(g.out[30:], clean.out[30:])
    assert torch.equal(g.out[10:, 4:], clean.out[10:, 4:])  # node j sees from P + j - 39 on
    if math.isnan(outlier):
        assert bool(g.out[:10, 4:].isnan().all())


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("far", [2.0 ** 6, 2.0 ** 12])
def test_one_scale_far_above_the_rest(kvq, fmt, far):  # noqa: F811
    """A node's value scale above all others: the rows that see it, within the bound."""
    b = TreeBatch([(300, 30), (2000, 16)], 8, 2, 128, fmt, PER_TOKEN_HEAD, seed=32)
    for L, n, i in ((300, 30, 0), (2000, 16, 1)):
        t = L - n + 4
        at = (int(b.bt[i, t // 16]), slice(None), t % 16)
        b.vs[at] *= far
        b.V[at] *= far
    g = OnGpu(kvq, b)
    g.call()
    check_scaled(g)


def check_scaled(g):
    """The batch's bound, and for per-(token, head) scales what 2^-24 of the row's largest weight is there: a weight enters
    as y s / sigma, sigma the power of two in [s_max, 2 s_max) of the scales seen, so it is off by 2^-24 sigma in y s, for
    every code of the dim that the row sees; the sum of weights is 1 at least."""
    b = g.b
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0
    ref, bound = b.reference()
    for i, (L, n) in enumerate(zip(b.lens, b.nodes)):
        t = torch.arange(L, device=b.dev)
        blk = b.bt[i][t // 16].long()
        s = b.vs[blk, :, t % 16].double()                                        # [L][hkv]
        codes = lib.decode(b.vc, b.fmt)[blk, :, t % 16].abs().sum(0)              # [hkv][dh]
        more = 2.0 ** -23 * s.amax(0)[:, None] * codes
        bound[int(b.cu[i]):int(b.cu[i + 1])] += more.repeat_interleave(b.hq // b.hkv, 0)
    err = (g.out.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("fmt,gran,dh", [(E4M3, PER_HEAD, 128), (E5M2, PER_HEAD, 64), (E4M3, PER_TOKEN_HEAD, 128), (BF16, PER_HEAD, 128),
                                         (BF16, PER_HEAD, 64)])
def test_bad_queries_stay_in_their_rows(kvq, fmt, gran, dh):  # noqa: F811
    """A NaN or an infinity in a query row is that row's output, whatever the keys' signs; the other rows keep their bits.
    A row that sees nothing stays zero."""
    b = TreeBatch([(300, 20), (2, 1), (2500, 16), (9, 9)], 8, 2, dh, fmt, gran, seed=41)
    b.bt[3] = -1
    clean = OnGpu(kvq, b)
    clean.call()
    rows = []
    for i, (row, head, d, x) in enumerate([(0, 1, 3, math.nan), (5, 0, dh - 1, math.inf), (19, 7, 0, -math.inf), (20, 0, 0, math.inf),
                                           (20, 1, 0, -math.inf), (20, 2, 1, math.inf), (20, 5, dh - 2, -math.inf), (30, 6, 9, math.inf),
                                           (36, 3, 17, -math.inf)]):
        b.q[row, head, d] = x
        rows.append((row, head))
    b.q[37:] = math.inf
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    assert int(g.st.item()) == int(clean.st.item()) == kvq.KVQ_DEV_BAD_BLOCK
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool, device="cuda")
    for row, head in rows:
        bad[row, head] = True
    assert bool(g.out[bad].isnan().all())
    assert torch.equal(g.out[~bad], clean.out[~bad]) and bool((g.out[37:] == 0).all())


@pytest.mark.parametrize("fmt", [E4M3, BF16])
@pytest.mark.parametrize("x", [math.inf, -math.inf])
def test_infinite_queries_against_keys_of_one_sign(kvq, fmt, x):  # noqa: F811
    """Logits that are all -inf (or all inf) are not a row that sees nothing."""
    b = TreeBatch([(70, 9), (300, 16)], 4, 2, 128, fmt, seed=42)
    b.kc[..., 5] = -1.0 if fmt == BF16 else 0xB8
    clean = OnGpu(kvq, b)
    clean.call()
    b.q[::2, 1, 5] = x
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0 and bool(g.out[::2, 1].isnan().all())
    g.out[::2, 1] = clean.out[::2, 1]
    assert torch.equal(g.out, clean.out)


def check_by_ties(g):
    """Every row, however large its logits: the output lies, dim by dim, between the least and the largest value of the keys
    whose logit may be the largest.

    A logit is off by D at most: over FP8 caches the query's parts leave 2^-17 of the row's largest value, times the key's
    magnitudes; binary32 sums 2^-19 of the sum of magnitudes.  A key more than 2 D + 40 below the largest logit has a weight of
    e^-40; 20000 of them and values 2^12 apart are below 2^-30 of the largest value that the row sees.  Beside that half a
    step of bf16, and 2^-11 and 2^-19 for weights and sums."""
    b = g.b
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0 and bool(g.out.isfinite().all())
    G, q = b.hq // b.hkv, b.query()
    for i, (L, n) in enumerate(zip(b.lens, b.nodes)):
        P, a = L - n, int(b.cu[i])
        t = torch.arange(L, device=b.dev)
        blk = b.bt[i][t // 16].long()
        see = torch.zeros(n, L, dtype=torch.bool)
        see[:, :P] = True
        for j in range(n):
            see[j, [P + k for k in lib.way_up(b.parents[i], j)]] = True
        see = see.cuda()
        for h in range(b.hkv):
            K, V = b.K[blk, h, t % 16], b.V[blk, h, t % 16]
            for j in range(n):
                qq = q[a + j, h * G:(h + 1) * G]                                     # [G][dh]
                x = (qq @ K.T / math.sqrt(b.dh)).masked_fill(~see[j], -math.inf)    # [G][L]
                D = 2.0 ** -19 * (qq.abs() @ K.abs().T).amax(1) / math.sqrt(b.dh)
                if b.fmt != BF16:
                    D = D + 2.0 ** -17 * qq.abs().amax(1) * K.abs().sum(1).max() / math.sqrt(b.dh)
                near = x >= (x.amax(1) - 2 * D - 40)[:, None]
                v = V[None].expand(G, -1, -1)
                lo = v.masked_fill(~near[..., None], math.inf).amin(1)
                hi = v.masked_fill(~near[..., None], -math.inf).amax(1)
                slack = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -19) * torch.maximum(lo.abs(), hi.abs()) + 2.0 ** -30 * V[see[j]].abs().amax()
                out = g.out[a + j, h * G:(h + 1) * G].double()
                assert bool(((out >= lo - slack) & (out <= hi + slack)).all()), (i, h, j)


@pytest.mark.parametrize("amp", [1e4, 1e30])
@pytest.mark.parametrize("fmt,gran", [(E4M3, PER_HEAD), (E5M2, PER_HEAD), (E4M3, PER_TOKEN_HEAD), (BF16, PER_HEAD)])
def test_large_queries_row_by_row(kvq, amp, fmt, gran):  # noqa: F811
    """Small trees, and long contexts that are cut into many pieces and merged."""
    for seqs in ([(300, 20), (40, 5)], [(20000, 5), (9000, 17)]):
        g = OnGpu(kvq, TreeBatch(seqs, 4, 2, 128, fmt, gran, amp=amp, seed=51))
        g.call()
        check_by_ties(g)


@pytest.mark.parametrize("fmt", [E4M3, BF16])
def test_small_queries_over_long_contexts(kvq, fmt):  # noqa: F811
    for amp in (1e-30, 1e-4):
        g = OnGpu(kvq, TreeBatch([(20000, 5), (9000, 17)], 4, 2, 128, fmt, amp=amp, seed=52))
        g.call()
        g.check()


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("small", [2.0 ** -17, 2.0 ** -16 * 0.75, 2.0 ** -15 * 1.3, 2.0 ** -9 * 1.01])
def test_small_query_values_beside_a_large_one(kvq, fmt, small):  # noqa: F811
    """127 equal values far below a row's first, which meets keys of 0: what the two E4M3 parts leave of them shows.

    The row's largest value is taken to 2^7 at least, where E4M3's least step is 2^-9: a value is off by half of it, 2^-17
    of the largest.  The logit is off by that times the key's magnitudes, and 2^-19 of itself; the weights by twice as much."""
    n, dh = 8, 128
    t = TreeBatch([(2 + n, n)], 4, 1, dh, fmt, PER_TENSOR, kind="forest", seed=61)
    K, V = torch.zeros(2 + n, dh), torch.zeros(2 + n, dh)
    K[1:2, 1:] = lib.TOP[fmt] if fmt == E4M3 else 512.0
    V[0], V[1] = -1.0, 1.0
    fill(t, K, V)
    q = torch.full((n, 4, dh), small)
    q[..., 0] = torch.linspace(1.0, 1.9, n)[:, None]
    t.q = q.to(torch.bfloat16).cuda()
    o = OnGpu(kvq, t)
    o.call()
    torch.cuda.synchronize()
    assert int(o.st.item()) == 0
    x = t.q.double() @ K[1].double().cuda() / math.sqrt(dh)
    a = torch.exp(x)  # the first token and the node itself weigh 1
    ref = (a - 1) / (a + 2)
    d = (2.0 ** -17 * t.q.double().amax(-1) * K[1].sum().item() + 2.0 ** -19 * x.abs()) / math.sqrt(dh) + 2.0 ** -19 * x.abs()
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -18 + 2 * d) * (a + 1) / (a + 2)
    err = (o.out.double() - ref[..., None]).abs()
    assert bool((err <= bound[..., None]).all()), float((err / bound[..., None]).max())


@pytest.mark.parametrize("dh", [64, 128])
def test_large_values_of_bf16_caches(kvq, dh):  # noqa: F811
    """V times 2^84 (values to 2^90) gives the outputs times 2^84, bit for bit: no sum leaves binary32."""
    b = TreeBatch([(9000, 20), (300, 40), (17, 17)], 8, 2, dh, BF16, seed=71)
    g = OnGpu(kvq, b)
    g.call()
    clean = g.out.clone()
    b.vc.copy_(torch.nan_to_num(b.vc.double()) * 2.0 ** 84)
    g.call()
    torch.cuda.synchronize()
    assert torch.equal(g.out.double(), clean.double() * 2.0 ** 84)


@pytest.mark.parametrize("fmt,gran,dh", [(E4M3, PER_HEAD, 128), (E5M2, PER_TOKEN_HEAD, 64), (BF16, PER_HEAD, 128)])
def test_bad_values_before_the_tree(kvq, fmt, gran, dh):  # noqa: F811
    """NaN and infinities in tokens that every row of a sequence sees, far from its tree: a value's in its own dim, a key's in
    its head's rows, nothing elsewhere."""
    b = TreeBatch([(3000, 20), (500, 30), (9000, 9)], 8, 2, dh, fmt, gran, seed=72)
    g = OnGpu(kvq, b)
    g.call()
    clean = g.out.clone()
    nan = math.nan if fmt == BF16 else 0x7F
    at = lambda i, t: (int(b.bt[i, t // 16]), t % 16)  # noqa: E731
    blk, s = at(0, 700)
    b.vc[blk, 1, s, 3] = nan
    blk, s = at(1, 100)
    b.kc[blk, 0, s, 5] = nan
    bad = torch.zeros(b.q.shape, dtype=torch.bool, device="cuda")
    bad[:20, 4:, 3] = True
    bad[20:50, :4] = True
    if fmt != E4M3:
        blk, s = at(2, 4000)
        b.vc[blk, 1, s, 9] = math.inf if fmt == BF16 else 0x7C
        bad[50:, 4:, 9] = True
    g.call()
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0
    assert bool(g.out[:50][bad[:50]].isnan().all()) and not bool(g.out[50:][bad[50:]].isfinite().any())
    assert torch.equal(g.out[~bad], clean[~bad])
