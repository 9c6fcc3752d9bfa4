"""Paths of the 4-bit cache's kernels that small batches do not take: more tokens than
the write's threads, the read's rules for many rows, shared-out keys of two-tile items."""
import numpy as np
import pytest
import torch

import fp4_testlib as f4
from test_gpu_fp4 import OnGpu, _pages_equal, dev, kvq, status  # noqa: F401

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
