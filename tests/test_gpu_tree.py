"""Attention over drafted trees against softmax attention in 64 bits over the same cache."""
import math

import pytest
import torch

import step_testlib as lib
from step_testlib import BF16, E4M3, E5M2, PER_HEAD, PER_TENSOR, PER_TOKEN_HEAD, OnGpu, TreeBatch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_paged_gb300 as m
    return m


def run(kvq, b, status=0, **kw):
    g = OnGpu(kvq, b)
    g.call(**kw)
    return g, g.check(status)


@pytest.mark.parametrize("fmt", [E4M3, E5M2, BF16])
@pytest.mark.parametrize("dh", [128, 64])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(20, 5)], [(128, 3), (129, 7)], [(500, 16), (16, 16), (77, 1)]], ids=str)
def test_small(kvq, fmt, dh, seqs):
    run(kvq, TreeBatch(seqs, 8, 2, dh, fmt, seed=len(seqs)))


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("fmt,dh", [(E4M3, 128), (E4M3, 64), (E5M2, 128), (BF16, 128), (BF16, 64)])
def test_groups_and_tiles(kvq, G, fmt, dh):
    """Trees of one row, of a tile and of several, ragged ones among them."""
    run(kvq, TreeBatch([(300, 130), (1000, 43), (64, 64), (9, 0), (700, 1)], 2 * G, 2, dh, fmt, seed=G))


@pytest.mark.parametrize("window", [1, 2, 5, 16, 63, 64, 200])
@pytest.mark.parametrize("fmt,dh", [(E4M3, 128), (BF16, 128), (E5M2, 64)])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_windows(kvq, window, fmt, dh, kind):
    run(kvq, TreeBatch([(400, 33), (90, 90), (33, 33), (2000, 5), (129, 128)], 4, 2, dh, fmt, window=window, kind=kind, seed=window))


@pytest.mark.parametrize("kind", ["chain", "star", "forest", "tree"])
def test_kinds_of_trees(kvq, kind):
    run(kvq, TreeBatch([(600, 256), (256, 256), (31, 30), (1024, 64)], 8, 4, 128, kind=kind))


def test_chain_without_parents(kvq):
    for window in (0, 20):
        b = TreeBatch([(600, 200), (33, 33), (1024, 7)], 8, 2, 128, kind="chain", window=window)
        g, _ = run(kvq, b, parents=None)
        out = g.out.clone()
        g.call()
        torch.cuda.synchronize()
        assert torch.equal(out, g.out)


@pytest.mark.parametrize("gran", [PER_TENSOR, PER_HEAD, PER_TOKEN_HEAD])
@pytest.mark.parametrize("qf8", [False, True])
@pytest.mark.parametrize("fmt,dh", [(E4M3, 128), (E5M2, 128), (E4M3, 64), (E5M2, 64)])
def test_scales(kvq, gran, qf8, fmt, dh):
    for window in (0, 50):
        run(kvq, TreeBatch([(900, 40), (130, 9), (16, 1)], 8, 2, dh, fmt, gran, qf8=qf8, seed=gran, window=window))


@pytest.mark.parametrize("fmt,dh", [(E4M3, 128), (E4M3, 64), (BF16, 128), (E5M2, 128)])
def test_long_context_is_shared_out(kvq, fmt, dh):
    run(kvq, TreeBatch([(20000, 17)], 8, 2, dh, fmt))
    run(kvq, TreeBatch([(9000, 64), (12000, 200)], 8, 1, dh, fmt))


def test_uneven_batches(kvq):
    """Many short sequences beside a long one, empty trees and lengths of all kinds."""
    g = torch.Generator().manual_seed(3)
    seqs = []
    for i in range(120):
        n = int(torch.randint(0, 12, (1,), generator=g))
        seqs.append((n + int(2.0 ** float(torch.rand(1, generator=g) * 10)), n))
    seqs[50] = (15000, 30)
    run(kvq, TreeBatch(seqs, 8, 2, 128, E4M3, seed=4))
    run(kvq, TreeBatch(seqs, 6, 2, 64, BF16, seed=5, window=300))


def test_more_sequences_than_plan_entries(kvq):
    seqs = [(1 + i % 40, (i % 5) * (i % 40 >= 4)) for i in range(2500)]
    run(kvq, TreeBatch(seqs, 2, 1, 64, E4M3, seed=6))


@pytest.mark.parametrize("amp", [1e-30, 1e-4, 1e4, 1e30])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_queries_of_any_magnitude(kvq, amp, fmt):
    """Small ones leave the mean; large ones a token's value (all but near ties of the largest logits)."""
    b = TreeBatch([(300, 20), (40, 5)], 4, 2, 128, fmt, amp=amp, seed=7)
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0 and bool(g.out.isfinite().all())
    if amp <= 1e-4:
        g.check()
    else:
        ref, _ = b.reference()
        far = ((g.out.double() - ref).abs().amax(-1) > 0.02 * ref.abs().amax(-1) + 0.01).double().mean()
        assert float(far) < 0.1


def test_wide_rows(kvq):
    """Rows whose values lie 2^20 apart: the small ones count for what they are next to the largest."""
    b = TreeBatch([(300, 20), (40, 5)], 4, 2, 128, E4M3, seed=8)
    b.q[..., ::3] *= 2.0 ** -20
    b.q[..., 1::3] *= 2.0 ** -9
    run(kvq, b)


@pytest.mark.parametrize("fmt", [E4M3, BF16])
def test_one_weight_far_above_the_rest(kvq, fmt):
    """A first token far above 20000 others whose weights, 2^-17 each, add up: they are not lost."""
    t = TreeBatch([(20000, 4)], 4, 1, 128, fmt, PER_TENSOR, seed=9, kind="chain")
    t.q.zero_()
    t.q[..., 0] = 1.0
    scale = (t.ks.item(), t.vs.item()) if t.ks is not None else (1.0, 1.0)
    k, v = torch.zeros(t.nb, 1, lib.BS, 128, device="cuda"), torch.full((t.nb, 1, lib.BS, 128), 2.0, device="cuda")
    blk = int(t.bt[0, 0])
    k[blk, 0, 0, 0] = 11.8 * math.sqrt(128)
    v[blk, 0, 0] = -1.0
    if t.ks is not None:  # codes up to 448 hold it
        t.ks.fill_(1.0)
        scale = (1.0, scale[1])
    for c, x, s in ((t.kc, k, scale[0]), (t.vc, v, scale[1])):
        c.copy_(x.to(torch.bfloat16) if fmt == BF16 else lib.encode(x / s, fmt))
    t.K, t.V = (lib.decode(c, fmt) * s for c, s in ((t.kc, scale[0]), (t.vc, scale[1])))
    run(kvq, t)


@pytest.mark.parametrize("fmt,dh", [(E4M3, 128), (E5M2, 128), (BF16, 128), (E4M3, 64), (BF16, 64)])
@pytest.mark.parametrize("window", [0, 40])
def test_nan_reaches_those_who_see_it(kvq, fmt, dh, window):
    """NaN in K and V of a node, and of a token at the window's edge: rows that do not see it are as without it."""
    b = TreeBatch([(200, 30), (90, 20)], 4, 2, dh, fmt, window=window, seed=10)
    clean = OnGpu(kvq, b)
    clean.call()
    torch.cuda.synchronize()
    P = 170
    spots = [(P + 4, b.vc, 3), (P + 9, b.kc, 7)] + ([(P - 33, b.vc, 1)] if window else [])
    for t, c, d in spots:
        c[int(b.bt[0, t // 16]), 1, t % 16, d] = math.nan if fmt == BF16 else 0x7F
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    assert torch.equal(g.out[:, :2], clean.out[:, :2]) and torch.equal(g.out[30:], clean.out[30:])
    for j in range(30):
        way = lib.way_up(b.parents[0], j)
        near = way[:window] if window else way
        first = max(0, P + len(way) - window) if window else 0
        sees_v, sees_k, sees_w = 4 in near, 9 in near, bool(window) and P - 33 >= first
        row = g.out[j, 2:]
        want = torch.zeros(dh, dtype=torch.bool, device="cuda")
        want[3] = want[3] | sees_v
        want[1] = want[1] | sees_w
        want |= sees_k
        assert bool((row.isnan() == want).all()), j
        if not (sees_v or sees_k or sees_w):
            assert torch.equal(row, clean.out[j, 2:])


def test_infinities_in_values(kvq):
    """A cache from elsewhere may hold E5M2 infinities: rows that see one are infinite there, the others do not change."""
    b = TreeBatch([(100, 30)], 2, 1, 128, E5M2, seed=11)
    clean = OnGpu(kvq, b)
    clean.call()
    t = 70 + 3
    b.vc[int(b.bt[0, t // 16]), 0, t % 16, 9] = 0x7C
    b.vc[int(b.bt[0, t // 16]), 0, t % 16, 70] = 0xFC
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    for j in range(30):
        sees = 3 in lib.way_up(b.parents[0], j)
        same = torch.ones(128, dtype=torch.bool, device="cuda")
        same[9] = same[70] = not sees
        assert torch.equal(g.out[j][:, same], clean.out[j][:, same])
        if sees:
            assert bool((g.out[j, :, 9] == math.inf).all() & (g.out[j, :, 70] == -math.inf).all())


@pytest.mark.parametrize("fmt,gran", [(E4M3, PER_HEAD), (E4M3, PER_TOKEN_HEAD), (BF16, PER_HEAD)])
def test_bad_pages_are_masked(kvq, fmt, gran):
    b = TreeBatch([(400, 20), (100, 9), (30, 30)], 4, 2, 128, fmt, gran, seed=12)
    b.bt[0, 3], b.bt[1, 0], b.bt[1, 6], b.bt[2, 0], b.bt[2, 1] = -1, b.nb, -7, 2 ** 31 - 1, -1  # the last: all that it has
    g, _ = run(kvq, b, kvq.KVQ_DEV_BAD_BLOCK)
    assert bool((g.out[29:] == 0).all())


def test_bad_lengths_and_offsets(kvq):
    b = TreeBatch([(200, 9), (50, 5), (60, 6), (70, 7), (300, 4)], 4, 2, 64, E4M3, seed=13)
    sl = b.sl.clone()
    sl[1], sl[2], sl[3] = 4, 10 ** 6, -5
    g = OnGpu(kvq, b)
    g.call(seq_lens=sl)
    torch.cuda.synchronize()
    assert int(g.st.item()) == kvq.KVQ_DEV_BAD_SEQLEN
    ref, bound = b.reference()
    good = (g.out.double() - ref).abs() <= bound
    assert bool((g.out[9:27] == 0).all()) and bool(good[:9].all()) and bool(good[27:].all())
    # offsets that are negative, fall, or pass the rows: those rows stay as they were
    for cu, wrong in (([-1, 9, 14, 20, 27, 31], slice(0, 9)), ([0, 9, 14, 20, 27, 99], slice(27, 31)), ([0, 9, 9, 5, 27, 31], slice(0, 0))):
        g = OnGpu(kvq, b)
        g.call(cu_q_lens=torch.tensor(cu, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert int(g.st.item()) & kvq.KVQ_DEV_BAD_QLEN
        assert bool((g.out[wrong] == 7).all())
        if wrong.stop:
            rest = torch.ones(31, dtype=torch.bool, device="cuda")
            rest[wrong] = False
            assert bool(((g.out.double() - ref).abs() <= bound)[rest].all())


def test_too_many_nodes(kvq):
    b = TreeBatch([(400, 257), (300, 256)], 2, 1, 64, E4M3, seed=14)
    g = OnGpu(kvq, b)
    g.call()
    torch.cuda.synchronize()
    assert int(g.st.item()) == kvq.KVQ_DEV_BAD_QLEN
    ref, bound = b.reference()
    assert bool((g.out[:257] == 7).all()) and bool(((g.out.double() - ref).abs() <= bound)[257:].all())


def test_bad_parents_count_as_none(kvq):
    b = TreeBatch([(100, 12)], 4, 2, 128, E4M3, seed=15)
    par = b.par.clone()
    par[3], par[5], par[7], par[0] = 3, 11, -2, 2 ** 31 - 1
    for j in (3, 5, 7, 0):
        b.parents[0][j] = -1
    run(kvq, b, kvq.KVQ_DEV_BAD_TREE, parents=par)


def test_rows_behind_the_last_sequence_stay(kvq):
    b = TreeBatch([(100, 12), (40, 4)], 4, 2, 128, E4M3, seed=16)
    q = torch.cat([b.q, torch.full((5, 4, 128), math.nan, dtype=torch.bfloat16, device="cuda")])
    out = torch.full_like(q, 7.0)
    par = torch.cat([b.par, torch.full((5,), 99, dtype=torch.int32, device="cuda")])
    g = OnGpu(kvq, b)
    g.call(q=q, out=out, parents=par)
    g.out = out[:16]
    g.check()
    assert bool((out[16:] == 7).all())


def test_nothing_to_do(kvq):
    b = TreeBatch([(100, 0), (40, 0)], 4, 2, 128, E4M3, seed=17)
    g = OnGpu(kvq, b)
    g.call()
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    g.call(q=q, out=out, parents=torch.zeros(3, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0 and bool((out == 7).all())


def test_same_bits_again_and_in_graphs(kvq):
    """Two captured graphs with a workspace each, replayed in turn and beside each other; another stream."""
    b, c = TreeBatch([(7000, 40), (200, 9)], 8, 2, 128, E4M3, seed=18), TreeBatch([(5000, 64)], 8, 2, 128, E5M2, seed=19)
    first = []
    for x in (b, c):
        g, _ = run(kvq, x)
        first.append(g.out.clone())
        for _ in range(3):
            g.call()
            torch.cuda.synchronize()
            assert torch.equal(g.out, first[-1])
    gs, graphs = [OnGpu(kvq, x) for x in (b, c)], []
    for g in gs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            g.call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for g in gs:
        g.out.fill_(7.0)
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for g, f in zip(gs, first):
        assert torch.equal(g.out, f) and int(g.st.item()) == 0
    gs[0].out.fill_(7.0)
    streams[0].wait_stream(torch.cuda.current_stream())
    gs[0].call(stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(gs[0].out, first[0])


def test_one_node_is_the_decode(kvq):
    """A tree of one node attends as kvq_decode_attn does."""
    b = TreeBatch([(100, 1), (1, 1), (3000, 1)], 8, 2, 128, E4M3, seed=20)
    run(kvq, b)
    out = torch.empty_like(b.q)
    kvq.kvq_decode_attn(b.q, b.kc, b.vc, b.bt, b.sl, None, b.ks, b.vs, b.gran, b.fmt, 0, kvq.new_workspace(3, 8, 2, 128), out)
    ref, bound = b.reference()
    torch.cuda.synchronize()
    assert bool(((out.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("fmt,gran", [(BF16, PER_HEAD), (E4M3, PER_TOKEN_HEAD), (E4M3, PER_HEAD)])
@pytest.mark.parametrize("dh", [128, 64])
def test_edges_behind_long_runs(kvq, fmt, gran, dh):
    """Edge blocks, whose V is looked at and cleared, behind many others of the same CTA: a V that is still to
    come into the slot before is not touched.  (Rings hold 4 to 16 blocks, and 6 are in flight.)"""
    seqs = [(700 + 226 * i, 30) for i in range(16)]
    g = OnGpu(kvq, TreeBatch(seqs, 28, 4, dh, fmt, gran, seed=dh))
    g.call()
    g.check()
    first = g.out.clone()
    for _ in range(30):
        g.out.fill_(7.0)
        g.call()
        assert torch.equal(g.out.view(torch.uint8), first.view(torch.uint8))
