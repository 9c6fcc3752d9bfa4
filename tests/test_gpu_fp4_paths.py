"""Paths of the 4-bit cache's kernels that small batches do not take: more tokens than
the write's threads, the read's rules for many rows, shared-out keys of two-tile items."""
import numpy as np
import pytest
import torch

import fp4_testlib as f4
from test_gpu_fp4 import OnGpu, _pages_equal, bits, dev, kvq, status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv,dh,tokens", [(8, 128, 5300), (40, 64, 1500), (40, 128, 1400), (7, 64, 12000)])
def test_write_more_tokens_than_threads(kvq, hkv, dh, tokens):  # noqa: F811
    """Every thread takes several tokens, with padding and bad slots among the later ones."""
    b = f4.Batch(hkv + dh, [tokens], hkv, hkv, dh)
    slots = b.slots.copy()
    slots[[0, tokens // 2, tokens - 1]] = -1
    _pages_equal(kvq, b.k, b.v, slots, b.nb, hkv, dh, b.ks, b.vs, b.gran, fill=0x5A)
    slots[[tokens - 2, tokens // 3]] = b.nb * 16, 1 << 50
    _pages_equal(kvq, b.k, b.v, slots, b.nb, hkv, dh, b.ks, b.vs, b.gran, want_status=kvq.KVQ_DEV_BAD_SLOT)


@pytest.mark.parametrize("rows", [1023, 1100, 65535, 66000])
@pytest.mark.parametrize("hkv,dh", [(8, 128), (1, 64), (3, 128)])
def test_read_many_rows(kvq, rows, hkv, dh):  # noqa: F811
    """Sequences of all lengths, empty ones among them, over shared pages."""
    b = f4.Batch(rows + hkv, [700], hkv, hkv, dh)
    K, V = b.pages()
    # the bf16 bits of each page's rows [blocks][16][hkv][dh], as binary32 products
    want = [f4.to_bf16((f4.unit_values(c).astype(np.float32) * s.reshape(1, hkv, 1, 1)).astype(np.float32)).transpose(0, 2, 1, 3)
            for c, s in ((K, b.ks), (V, b.vs))]
    r, n = np.random.default_rng(rows), []
    while sum(n) < rows:
        n.append(min(int(r.integers(0, 500)) * int(r.random() < 0.8), rows - sum(n)))
    n.append(0)
    B = len(n)
    starts = r.integers(0, 200, B).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    seq = np.repeat(np.arange(B), n)
    pos = np.arange(rows) - cu[seq] + starts[seq]
    blk = b.table[0, pos // 16].astype(np.int64)
    ko = torch.full((rows + 2, hkv, dh), 2.0, dtype=torch.bfloat16, device="cuda")
    vo, st = ko.clone(), status()
    kvq.kvq_fp4_read(dev(K), dev(V), dev(np.repeat(b.table, B, 0)), dev(starts), dev(cu), dev(b.ks), dev(b.vs), b.gran,
                     ko, vo, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    at = dev(blk), dev(pos % 16)
    for out, w in ((ko, want[0]), (vo, want[1])):
        assert torch.equal(out[:rows].view(torch.int16), dev(w)[at].view(torch.int16))
        assert bool((out[rows:] == 2).all())


@pytest.mark.parametrize("B,chunk,hq,dh", [(160, 20, 8, 64), (160, 33, 4, 128), (80, 70, 4, 128)])
def test_prefill_two_tiles_shared_out(kvq, B, chunk, hq, dh):  # noqa: F811
    """More items of two tiles than SMs; the last ones, over long sequences, share their keys out."""
    long = 6300
    b = f4.Batch(B + dh, [long], hq, 1, dh)
    b.table = np.repeat(b.table, B, 0)
    counts = [max(1, chunk - i % 7) for i in range(B)]
    counts[-1] = chunk
    b.lens = np.array([counts[i] + 11 * i % 90 if i < B - 9 else long - 400 * (B - 1 - i) // 9 for i in range(B)], np.int32)
    for window, sinks in ((0, 0), (6200, 5)):
        g = OnGpu(kvq, b, counts)
        g.prefill(window, sinks)
        g.check(window, sinks, "first")
        first = g.out.clone()
        g.prefill(window, sinks)
        torch.cuda.synchronize()
        assert torch.equal(first, g.out)


@pytest.mark.parametrize("cu", [[0, 5, 14], [0, 8, 5], [-2, 3, 10], [-(1 << 31), (1 << 31) - 1, 10], [0, 4, 4 + (1 << 30)]])
def test_prefill_bad_chunk_bounds(kvq, cu):  # noqa: F811
    """Chunks that end past the queries, or whose bounds decrease or are negative, are
    reported, and their rows left alone; the others are right."""
    b = f4.Batch(3, [40, 33], 8, 2, 64)
    g = OnGpu(kvq, b, [5, 5])
    cu = np.array(cu, np.int64)
    bad = (cu[:-1] < 0) | (cu[1:] < cu[:-1]) | (cu[1:] > 10)
    g.dcu = dev(cu.astype(np.int32))
    g.prefill(max_q=10)
    torch.cuda.synchronize()
    assert int(g.st.item()) == kvq.KVQ_DEV_BAD_QLEN
    # the good chunks alone, beside sequences without queries
    mine = np.zeros(10, bool)
    for s in np.nonzero(~bad)[0]:
        lens = np.where(np.arange(2) == s, b.lens, 0)
        one = np.where(np.arange(3) <= s, 0, cu[s + 1] - cu[s])
        want, tol = f4.attention(g.q[cu[s]:cu[s + 1]], g.K, g.V, b.ks, b.vs, b.table, lens, one, 0, 0)
        f4.check(bits(g.out[cu[s]:cu[s + 1]]), want, tol, f"sequence {s}")
        mine[cu[s]:cu[s + 1]] = True
    assert bool((g.out[torch.from_numpy(~mine).cuda()] == 7).all())


def test_prefill_bound_of_zero(kvq):  # noqa: F811
    """No queries at all are fine (the rows are padding); any chunk is past the bound."""
    b = f4.Batch(4, [40, 33], 8, 2, 64)
    g = OnGpu(kvq, b, [5, 5])
    for cu, want in (([0, 0, 0], 0), ([0, 0, 1], kvq.KVQ_DEV_BAD_QLEN), ([0, 10, 10], kvq.KVQ_DEV_BAD_QLEN)):
        g.st.zero_()
        g.dcu = dev(np.array(cu, np.int32))
        g.prefill(max_q=0)
        torch.cuda.synchronize()
        assert int(g.st.item()) == want
        assert bool((g.out == 7).all())


def test_prefill_of_no_queries(kvq):  # noqa: F811
    """A step in which no sequence has new tokens, with empty tensors."""
    b = f4.Batch(5, [40, 33], 8, 2, 64)
    g = OnGpu(kvq, b, [0, 0])
    for max_q in (0, 16):
        g.prefill(max_q=max_q)
    torch.cuda.synchronize()
    assert int(g.st.item()) == 0


@pytest.mark.parametrize("lens,counts,hq,hkv,dh", [([2500], [3], 32, 8, 128), ([5000], [40], 16, 4, 64), ([2300] * 20, [2] * 20, 8, 8, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 7)])
def test_nan_in_shared_out_keys(kvq, lens, counts, hq, hkv, dh, window, sinks):  # noqa: F811
    """NaN keys and values in tokens of one piece of a sequence reach the rows that see them
    through the merge, and no others; a sequence that is NaN alone, too."""
    b = f4.Batch(len(lens) + dh + window, lens, hq, hkv, dh)
    b.k[2, 0, 3] = b.v[5, 1, 40] = b.v[1200, 2, 17] = b.k[lens[0] - 2, 3, 50] = 0x7FC0
    if len(lens) > 1:
        b.k[lens[0]:2 * lens[0], 4, 0] = 0x7FC0
    for n, call in (([1] * len(lens), "decode"), (counts, "prefill")):
        g = OnGpu(kvq, b, n)
        getattr(g, call)(window, sinks)
        g.check(window, sinks, call)
        assert bool(torch.isnan(g.out.float()).any()) and not bool(torch.isnan(g.out.float()).all())
