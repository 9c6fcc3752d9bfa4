"""The 4-bit cache's kernels against plain numpy: pages bit for bit, gathered
rows bit for bit, attention within the bound that fp4_testlib.attention
derives."""
import numpy as np
import pytest
import torch

import fp4_testlib as f4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import fp8_quantized_paged_gb300 as m
    return m


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(a).cuda()


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def workspace(kvq, B, hq, hkv, dh):
    """NaN bytes everywhere but the counters, which start at zero."""
    ws = kvq.new_fp4_workspace(B, hq, hkv, dh)
    ws.fill_(0xFF)
    ws[:kvq.KVQ_WS_COUNTER_BYTES].zero_()
    return ws


class OnGpu:
    """A Batch's pages and queries on the device."""

    def __init__(self, kvq, b, counts):
        self.kvq, self.b = kvq, b
        self.K, self.V = b.pages()
        self.q, self.cu = b.queries(counts)
        self.kc, self.vc, self.dq = dev(self.K), dev(self.V), dev(self.q)
        self.bt, self.sl, self.dcu = dev(b.table), dev(b.lens), dev(self.cu)
        self.ks, self.vs = dev(b.ks), dev(b.vs)
        self.ws = workspace(kvq, len(b.lens), b.hq, b.hkv, b.dh)
        self.out = torch.full((max(1, self.q.shape[0]), b.hq, b.dh), 7.0, dtype=torch.bfloat16, device="cuda")[:self.q.shape[0]]
        self.st = status()

    def decode(self, window=0, sinks=0, stream=None):
        self.kvq.kvq_fp4_decode_attn(self.dq, self.kc, self.vc, self.bt, self.sl, self.ks, self.vs, self.b.gran,
                                     window, sinks, self.ws, self.out, dev_status=self.st, stream=stream)

    def prefill(self, window=0, sinks=0, max_q=None, stream=None):
        n = int(np.diff(self.cu).max()) if max_q is None else max_q
        self.kvq.kvq_fp4_prefill_attn(self.dq, self.dcu, n, self.kc, self.vc, self.bt, self.sl, self.ks, self.vs,
                                      self.b.gran, window, sinks, self.ws, self.out, dev_status=self.st, stream=stream)

    def check(self, window=0, sinks=0, what="", status=0, twice=True):
        want, tol = f4.attention(self.q, self.K, self.V, self.b.ks, self.b.vs, self.b.table, self.b.lens, self.cu, window, sinks)
        torch.cuda.synchronize()
        assert int(self.st.item()) == status, what
        f4.check(bits(self.out), want, tol, what)
        n = self.kvq.KVQ_WS_COUNTER_BYTES
        assert not self.ws[:n].any(), f"{what}: counters left behind"


# ------------------------------------------------------------------ write

def _pages_equal(kvq, k, v, slots, nb, hkv, dh, ks, vs, gran, fill=0, want_status=0, stride=None):
    K, V = f4.new_cache(nb, hkv, dh, fill), f4.new_cache(nb, hkv, dh, fill)
    kc, vc, st = dev(K), dev(V), status()
    dk, dv = dev(k), dev(v)
    if stride:
        n = len(slots)
        big = torch.full((n, 2, stride), 9.0, dtype=torch.bfloat16, device="cuda")
        dk2 = big[:, 0, :hkv * dh].view(n, hkv, dh) if n == 0 else big[:, 0, :hkv * dh].unflatten(1, (hkv, dh))
        dv2 = big[:, 1, :hkv * dh].unflatten(1, (hkv, dh))
        dk2.copy_(dk)
        dv2.copy_(dv)
        dk, dv = dk2, dv2
    kvq.kvq_fp4_write(dk, dv, dev(np.asarray(slots, np.int64)), kc, vc, dev(ks), dev(vs), gran, dev_status=st)
    f4.write(k, slots, K, ks)
    f4.write(v, slots, V, vs)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    assert np.array_equal(kc.cpu().numpy(), K)
    assert np.array_equal(vc.cpu().numpy(), V)


@pytest.mark.parametrize("hkv,dh", [(1, 64), (2, 64), (3, 128), (8, 128), (40, 64)])
@pytest.mark.parametrize("lens", [[1], [5, 0, 33], [200, 17]])
@pytest.mark.parametrize("per_head", [True, False])
def test_write_pages(kvq, hkv, dh, lens, per_head):
    b = f4.Batch(hkv * dh + len(lens), lens, hkv, hkv, dh, per_head)
    _pages_equal(kvq, b.k, b.v, b.slots, b.nb, hkv, dh, b.ks, b.vs, b.gran, fill=0x5A)


def test_write_row_distance_padding_and_bad_slots(kvq):
    b = f4.Batch(3, [40], 4, 4, 64)
    slots = b.slots.copy()
    slots[[0, 7, 39]] = -1, -(1 << 40), -5
    _pages_equal(kvq, b.k, b.v, slots, b.nb, 4, 64, b.ks, b.vs, b.gran, stride=4 * 64 + 24)
    slots[3] = b.nb * 16
    slots[4] = 1 << 40
    _pages_equal(kvq, b.k, b.v, slots, b.nb, 4, 64, b.ks, b.vs, b.gran, want_status=kvq.KVQ_DEV_BAD_SLOT)


@pytest.mark.parametrize("scale", [1e-40, 2.0 ** -120, 1e-25, 1e-10, 1.0, 3.14159, 1e10, 1e30, 3e38])
def test_write_all_magnitudes(kvq, scale):
    """Every finite bf16 magnitude class, infinities, NaN, signed zeros and
    subnormals, each block of its own magnitude, over small and large scales."""
    r = np.random.default_rng(5)
    n, hkv, dh = 64, 2, 128
    e = r.integers(0, 255, (n, hkv, dh // 16, 1))
    e = np.clip(e - r.integers(0, 6, (n, hkv, dh // 16, 16)), 0, 254)
    k = ((r.integers(0, 2, e.shape) << 15) | (e << 7) | r.integers(0, 128, e.shape)).astype(np.uint16).reshape(n, hkv, dh)
    v = k[::-1].copy()
    v[1, 0, 5] = 0x7F80                 # inf
    v[2, 0, 5] = 0xFF80
    v[3, 1, 17] = 0x7FC0                # NaN
    v[4] = 0x8000                       # -0
    v[5] = 0
    slots = np.arange(n, dtype=np.int64)
    s = np.array([scale, min(3e38, scale * 1.37)], np.float32)
    _pages_equal(kvq, k, v, slots, 4, hkv, dh, s, s[::-1].copy(), f4.PER_HEAD)


def test_write_every_significand(kvq):
    """All 128 bf16 significands against many scales: quotients at and beside ties."""
    r = np.random.default_rng(6)
    m = np.arange(128)
    for seed in range(8):
        x = np.stack([r.permutation(m) for _ in range(32)]).reshape(32, 2, 64)
        e = r.integers(120, 131, (32, 2, 64))
        k = ((r.integers(0, 2, x.shape) << 15) | (e << 7) | x).astype(np.uint16)
        s = np.array([2.0 ** -r.integers(5, 12), r.uniform(0.001, 0.1)], np.float32)
        _pages_equal(kvq, k, k[:, ::-1].copy(), np.arange(32), 2, 2, 64, s, s, f4.PER_HEAD)


def test_write_nothing(kvq):
    b = f4.Batch(4, [5], 2, 2, 64)
    kc = dev(f4.new_cache(2, 2, 64, 3))
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    kvq.kvq_fp4_write(e, e, torch.empty(0, dtype=torch.int64, device="cuda"), kc, kc.clone(), dev(b.ks), dev(b.vs), b.gran)
    torch.cuda.synchronize()
    assert bool((kc == 3).all())


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("hkv,dh", [(1, 128), (3, 64), (8, 128)])
@pytest.mark.parametrize("per_head", [True, False])
def test_read_rows(kvq, hkv, dh, per_head):
    b = f4.Batch(7, [37, 0, 1, 64, 129], hkv, hkv, dh, per_head)
    K, V = b.pages()
    starts = np.array([5, 0, 0, 63, 16], np.int32)
    n = np.array([32, 0, 1, 1, 100])
    for st in (starts, None):
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        rows = int(cu[-1]) + 3
        big = torch.full((rows, hkv * dh + 8), 2.0, dtype=torch.bfloat16, device="cuda")
        ko = big[:, :hkv * dh].unflatten(1, (hkv, dh))
        vo = torch.full_like(big, 2.0)[:, :hkv * dh].unflatten(1, (hkv, dh))
        w = status()
        kvq.kvq_fp4_read(dev(K), dev(V), dev(b.table), None if st is None else dev(st), dev(cu), dev(b.ks), dev(b.vs),
                         b.gran, ko, vo, dev_status=w)
        torch.cuda.synchronize()
        assert int(w.item()) == 0
        two = int(f4.to_bf16(np.array([2.0]))[0])
        want = f4.read(K, b.ks, b.table, st, cu, rows, two), f4.read(V, b.vs, b.table, st, cu, rows, two)
        assert np.array_equal(bits(ko.contiguous()), want[0]) and np.array_equal(bits(vo.contiguous()), want[1])
        assert bool((big[:, hkv * dh:] == 2).all())


def test_read_bad_pages_and_positions(kvq):
    b = f4.Batch(8, [48, 48], 2, 2, 64)
    K, V = b.pages()
    table = b.table.copy()
    table[0, 1], table[1, 0] = b.nb, -3
    cu = np.array([0, 48, 60], np.int32)
    starts = np.array([0, 40], np.int32)  # the second runs past its table
    ko = torch.full((60, 2, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    vo, w = ko.clone(), status()
    kvq.kvq_fp4_read(dev(K), dev(V), dev(table), dev(starts), dev(cu), dev(b.ks), dev(b.vs), b.gran, ko, vo, dev_status=w)
    torch.cuda.synchronize()
    assert int(w.item()) == kvq.KVQ_DEV_BAD_BLOCK | kvq.KVQ_DEV_BAD_SEQLEN
    assert np.array_equal(bits(ko), f4.read(K, b.ks, table, starts, cu, 60))
    assert np.array_equal(bits(vo), f4.read(V, b.vs, table, starts, cu, 60))


def test_read_nan_block(kvq):
    b = f4.Batch(9, [16], 1, 1, 64)
    b.k[3, 0, 20] = 0x7FC0
    K, V = b.pages()
    ko = torch.zeros((16, 1, 64), dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    kvq.kvq_fp4_read(dev(K), dev(V), dev(b.table), None, dev(np.array([0, 16], np.int32)), dev(b.ks), dev(b.vs), b.gran, ko, vo)
    nan = torch.isnan(ko.cpu())
    assert bool(nan[3, 0, 16:32].all()) and int(nan.sum()) == 16 and not bool(torch.isnan(vo).any())


# ------------------------------------------------------------------ decode

MASKS = [(0, 0), (1, 0), (1, 1), (5, 3), (16, 4), (17, 16), (40, 33), (1000, 20)]


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (4, 2), (6, 2), (8, 2), (5, 1), (12, 2), (7, 1), (16, 2)])
def test_decode_groups(kvq, hq, hkv, dh):
    b = f4.Batch(hq * dh, [1, 16, 100, 37, 0, 333], hq, hkv, dh, per_head=hq % 2 == 0)
    g = OnGpu(kvq, b, [1] * 6)
    g.decode()
    g.check(what="decode")


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("dh", [64, 128])
def test_decode_masks(kvq, window, sinks, dh):
    b = f4.Batch(window + sinks, [1, 2, 15, 16, 17, 31, 48, 50, 129, 400], 8, 2, dh)
    g = OnGpu(kvq, b, [1] * 10)
    g.decode(window, sinks)
    g.check(window, sinks, "decode")


@pytest.mark.parametrize("lens,hq,hkv,dh", [
    ([5000], 32, 8, 128), ([9001], 8, 1, 128), ([7777], 16, 16, 64), ([3000, 1, 0, 2999], 28, 4, 128),
    ([1200, 3, 640, 640, 77, 1111, 16, 900], 8, 2, 64), ([2] * 300, 4, 4, 64), ([70] * 90, 16, 8, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
def test_decode_splits(kvq, lens, hq, hkv, dh, window, sinks):
    """Sequences cut over many blocks, and many sequences to one; the call again
    gives the same bits."""
    b = f4.Batch(len(lens), lens, hq, hkv, dh)
    g = OnGpu(kvq, b, [1] * len(lens))
    g.decode(window, sinks)
    g.check(window, sinks, "first")
    first = g.out.clone()
    g.out.fill_(3.0)
    g.decode(window, sinks)
    torch.cuda.synchronize()
    assert torch.equal(first, g.out)


@pytest.mark.parametrize("lens,hq,hkv,dh", [
    ([2300] * 20, 8, 8, 128), ([1700] * 40, 16, 8, 64), ([2100, 5, 1900, 640] * 8, 8, 4, 128),
    ([3100] * 16, 12, 6, 64), ([900, 4000, 17, 2500] * 5, 64, 8, 128)])
def test_decode_long_runs(kvq, lens, hq, hkv, dh):
    """Runs of many units per block, of 8, 4 and 2 heads each: the rings of shared pages
    go round several times."""
    b = f4.Batch(len(lens) + hkv, lens, hq, hkv, dh)
    g = OnGpu(kvq, b, [1] * len(lens))
    g.decode()
    g.check(what="first")
    first = g.out.clone()
    for _ in range(5):
        g.out.fill_(3.0)
        g.decode()
        torch.cuda.synchronize()
        assert torch.equal(first, g.out)


def test_decode_one_wide_query(kvq):
    """Logits up to hundreds (one token takes all) and queries of 1e-30 and 1e30."""
    b = f4.Batch(11, [300, 64], 8, 2, 128, amp=8.0)
    g = OnGpu(kvq, b, [1, 1])
    q = f4.bf16_to_f32(g.q).copy()
    q[0, 0] *= 40
    q[0, 1] *= 1e-30
    q[1, 2] *= 1e-30
    q[1, 3] = 0
    g.q = f4.to_bf16(q)
    g.dq = dev(g.q)
    g.decode()
    g.check(what="wide")


def test_decode_bad_blocks_and_lengths(kvq):
    b = f4.Batch(12, [100, 100, 40, 16], 8, 2, 128)
    g = OnGpu(kvq, b, [1] * 4)
    b.table[0, 2], b.table[1, 6], b.table[3, 0] = b.nb, -1, 1 << 30
    g.bt = dev(b.table)
    g.decode()
    g.check(what="bad blocks", status=kvq.KVQ_DEV_BAD_BLOCK)
    b.lens[2], b.lens[3] = b.table.shape[1] * 16 + 1, -4
    g.sl = dev(b.lens)
    g.st.zero_()
    g.decode()
    g.check(what="bad lengths", status=kvq.KVQ_DEV_BAD_BLOCK | kvq.KVQ_DEV_BAD_SEQLEN)


def test_decode_nan_reaches_its_head_only(kvq):
    b = f4.Batch(13, [50, 20], 4, 2, 64)
    b.k[30, 0, 3] = 0x7FC0       # a key of KV head 0: its two query heads are NaN
    b.v[60, 1, 40] = 0x7FC0      # a value: one block of dims of KV head 1's query heads
    g = OnGpu(kvq, b, [1, 1])
    g.decode()
    torch.cuda.synchronize()
    got = np.isnan(f4.bf16_to_f32(bits(g.out)))
    want = np.zeros_like(got)
    want[0, 0:2] = True
    want[1, 2:4, 32:48] = True
    assert np.array_equal(got, want)
    # tokens [40, 50) and [10, 20): the key at 30 is out of sight, the value at
    # position 10 just in it, and with one token less out of it
    want[0] = False
    for window, seen in ((10, want), (9, np.zeros_like(want))):
        g.decode(window)
        torch.cuda.synchronize()
        assert np.array_equal(np.isnan(f4.bf16_to_f32(bits(g.out))), seen)
        g.check(window, 0, "window")


# ------------------------------------------------------------------ prefill

@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (3, 1), (8, 2), (10, 2), (6, 1), (14, 2), (8, 1)])
def test_prefill_groups(kvq, hq, hkv, dh):
    b = f4.Batch(hq + dh, [70, 33, 5, 0, 150], hq, hkv, dh, per_head=hq % 2 == 0)
    g = OnGpu(kvq, b, [70, 1, 5, 0, 40])
    g.prefill()
    g.check(what="prefill")


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("dh", [64, 128])
def test_prefill_masks(kvq, window, sinks, dh):
    b = f4.Batch(window + sinks + 1, [1, 17, 90, 260, 400], 8, 2, dh)
    g = OnGpu(kvq, b, [1, 17, 30, 260, 3])
    g.prefill(window, sinks)
    g.check(window, sinks, "prefill")


@pytest.mark.parametrize("lens,counts,hq,hkv,dh", [
    ([2500], [1], 32, 8, 128), ([2500], [3], 32, 8, 128), ([3001, 1700], [9, 4], 16, 4, 128),
    ([2100], [600], 4, 1, 128), ([1000] * 6, [64, 7, 1, 100, 33, 16], 8, 2, 64),
    ([4000], [130], 8, 8, 64), ([1500, 20, 800], [150, 20, 90], 28, 4, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 20)])
def test_prefill_chunks(kvq, lens, counts, hq, hkv, dh, window, sinks):
    b = f4.Batch(sum(lens), lens, hq, hkv, dh)
    g = OnGpu(kvq, b, counts)
    g.prefill(window, sinks)
    g.check(window, sinks, "first")
    first = g.out.clone()
    g.out.fill_(3.0)
    g.prefill(window, sinks)
    torch.cuda.synchronize()
    assert torch.equal(first, g.out)


@pytest.mark.parametrize("lens,counts,hkv,dh,window,sinks", [
    ([260, 150], [233, 150], 4, 128, 16, 1), ([166, 196], [166, 186], 1, 64, 16, 5000), ([595], [255], 2, 128, 300, 17),
    ([400], [400], 2, 64, 40, 20)])
def test_prefill_second_tile_still_sees_the_first_tokens(kvq, lens, counts, hkv, dh, window, sinks):
    """A tile whose window has left the first pages, beside one whose first row sees
    every token there is."""
    b = f4.Batch(22 + dh, lens, hkv, hkv, dh)
    g = OnGpu(kvq, b, counts)
    g.prefill(window, sinks)
    g.check(window, sinks, "prefill")


@pytest.mark.parametrize("dh,longest_last", [(64, True), (64, False), (128, True)])
def test_prefill_more_items_than_sms(kvq, dh, longest_last):
    """160 sequences on shared pages: a whole wave, and a rest whose keys are shared out
    where they are many."""
    b = f4.Batch(21 + dh, [6300], 8, 1, dh)
    b.table = np.repeat(b.table, 160, 0)
    b.lens = (300 + 37 * np.arange(160)[:: 1 if longest_last else -1]).astype(np.int32)
    g = OnGpu(kvq, b, [1 + i % 3 for i in range(160)])
    g.prefill()
    g.check(what="first")
    first = g.out.clone()
    g.prefill()
    torch.cuda.synchronize()
    assert torch.equal(first, g.out)


def test_prefill_bad_blocks_lengths_and_rows_behind(kvq):
    b = f4.Batch(15, [100, 100, 40, 16], 8, 2, 128)
    g = OnGpu(kvq, b, [20, 100, 10, 16])
    b.table[0, 2], b.table[1, 0], b.table[3, 0] = b.nb, -1, 1 << 30
    b.lens[2] = 9                           # shorter than its chunk
    g.bt, g.sl = dev(b.table), dev(b.lens)
    g.dq = torch.cat([g.dq, g.dq[:5]])      # rows behind the last sequence
    big = torch.full((g.dq.shape[0], 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, g.out = g.out, big
    g.prefill()
    g.out = big[:out.shape[0]]
    g.check(what="bad", status=kvq.KVQ_DEV_BAD_BLOCK | kvq.KVQ_DEV_BAD_SEQLEN)
    assert bool((big[out.shape[0]:] == 7).all())


def test_prefill_nan_only_where_seen(kvq):
    """NaN keys and values in tokens that a row does not see (later ones, ones before
    its window, ones between the first tokens and the window) leave it alone."""
    b = f4.Batch(18, [300, 150], 8, 2, 128)
    b.k[200, 0, 3] = b.k[310, 1, 90] = 0x7FC0
    b.v[250, 1, 40] = b.v[3, 0, 127] = b.v[420, 0, 0] = 0x7FC0
    for window, sinks in ((0, 0), (40, 0), (40, 5), (40, 2)):
        g = OnGpu(kvq, b, [140, 150])
        g.prefill(window, sinks)
        g.check(window, sinks, f"{window} {sinks}")


def test_prefill_chunk_longer_than_its_bound(kvq):
    b = f4.Batch(16, [600], 4, 1, 128)
    g = OnGpu(kvq, b, [600])
    g.prefill(max_q=100)
    torch.cuda.synchronize()
    assert int(g.st.item()) == kvq.KVQ_DEV_BAD_QLEN
    want, tol = f4.attention(g.q, g.K, g.V, b.ks, b.vs, b.table, b.lens, g.cu, 0, 0)
    f4.check(bits(g.out)[:100], want[:100], tol[:100], "rows within the bound")
    assert bool((g.out[512:] == 7).all())


def test_prefill_is_decode_for_one_query(kvq):
    b = f4.Batch(17, [33, 700, 16], 16, 2, 128)
    g = OnGpu(kvq, b, [1, 1, 1])
    for w, s in ((0, 0), (100, 7)):
        g.decode(w, s)
        g.check(w, s, "decode")
        g.out.zero_()
        g.prefill(w, s)
        g.check(w, s, "prefill")


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_generation(kvq, window, sinks):
    """Two prompts written and prefilled in chunks, then decoded token by token, on
    one workspace, and read back: every step as plain numpy has it."""
    hq, hkv, dh = 8, 2, 128
    full = f4.Batch(20, [90, 61], hq, hkv, dh, extra=0)
    q, cu = full.queries([90, 61])
    K, V = f4.new_cache(full.nb, hkv, dh, 0x7F), f4.new_cache(full.nb, hkv, dh, 0x7F)
    kc, vc, ks, vs, bt = dev(K), dev(V), dev(full.ks), dev(full.vs), dev(full.table)
    ws, st = workspace(kvq, 2, hq, hkv, dh), status()
    first = np.array([0, 90])
    done = np.array([0, 0])
    for counts in ([30, 7], [17, 40], [40, 10], [1, 1], [1, 1], [1, 1], [0, 1]):
        idx = np.concatenate([first[b] + done[b] + np.arange(counts[b]) for b in range(2)])
        done = done + counts
        lens, ccu = done.astype(np.int32), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        kvq.kvq_fp4_write(dev(full.k[idx]), dev(full.v[idx]), dev(full.slots[idx]), kc, vc, ks, vs, full.gran, dev_status=st)
        f4.write(full.k[idx], full.slots[idx], K, full.ks)
        f4.write(full.v[idx], full.slots[idx], V, full.vs)
        out = torch.zeros((len(idx), hq, dh), dtype=torch.bfloat16, device="cuda")
        want, tol = f4.attention(q[idx], K, V, full.ks, full.vs, full.table, lens, ccu, window, sinks)
        kvq.kvq_fp4_prefill_attn(dev(q[idx]), dev(ccu), max(counts), kc, vc, bt, dev(lens), ks, vs, full.gran, window, sinks, ws, out, dev_status=st)
        f4.check(bits(out), want, tol, f"prefill {counts}")
        if counts == [1, 1]:
            kvq.kvq_fp4_decode_attn(dev(q[idx]), kc, vc, bt, dev(lens), ks, vs, full.gran, window, sinks, ws, out, dev_status=st)
            f4.check(bits(out), want, tol, "decode")
    assert np.array_equal(kc.cpu().numpy(), K) and np.array_equal(vc.cpu().numpy(), V)
    ko = torch.zeros((151, hkv, dh), dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    rcu = np.array([0, 90, 151], np.int32)
    kvq.kvq_fp4_read(kc, vc, bt, None, dev(rcu), ks, vs, full.gran, ko, vo, dev_status=st)
    assert np.array_equal(bits(ko), f4.read(K, full.ks, full.table, None, rcu, 151))
    assert int(st.item()) == 0


def test_captured_step(kvq):
    """write, decode, prefill and read captured into one graph and replayed on
    changed inputs."""
    b = f4.Batch(21, [500, 31], 8, 2, 128)
    g = OnGpu(kvq, b, [1, 1])
    ko = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    last = np.array([499, 530])
    starts, rcu = dev(np.array([499, 30], np.int32)), dev(np.array([0, 1, 2], np.int32))
    k, v, slots = dev(b.k[last]), dev(b.v[last]), dev(b.slots[last])
    out2 = torch.zeros_like(g.out)

    def step():
        kvq.kvq_fp4_write(k, v, slots, g.kc, g.vc, g.ks, g.vs, b.gran, dev_status=g.st)
        g.decode(64, 4)
        kvq.kvq_fp4_prefill_attn(g.dq, g.dcu, 1, g.kc, g.vc, g.bt, g.sl, g.ks, g.vs, b.gran, 64, 4, g.ws, out2, dev_status=g.st)
        kvq.kvq_fp4_read(g.kc, g.vc, g.bt, starts, rcu, g.ks, g.vs, b.gran, ko, vo, dev_status=g.st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        r = np.random.default_rng(seed)
        kb, vb = (f4.to_bf16(r.standard_normal((2, 2, 128))) for _ in range(2))
        qb = f4.to_bf16(r.standard_normal((2, 8, 128)))
        k.copy_(dev(kb))
        v.copy_(dev(vb))
        g.dq.copy_(dev(qb))
        g.q = qb
        f4.write(kb, b.slots[last], g.K, b.ks)
        f4.write(vb, b.slots[last], g.V, b.vs)
        graph.replay()
        g.check(64, 4, f"replay {seed}")
        want, tol = f4.attention(qb, g.K, g.V, b.ks, b.vs, b.table, b.lens, g.cu, 64, 4)
        f4.check(bits(out2), want, tol, "prefill")
        assert np.array_equal(bits(ko), f4.read(g.K, b.ks, b.table, [499, 30], [0, 1, 2], 2))


def test_two_streams(kvq):
    """Two batches at once, each on its stream with its own workspace, the caller's
    current stream a third."""
    gs = [OnGpu(kvq, f4.Batch(30 + i, [1500, 900 + i], 8, 2, 128), [1, 1]) for i in range(2)]
    hs = [OnGpu(kvq, f4.Batch(40 + i, [400, 300 + i], 8, 2, 64), [100, 30]) for i in range(2)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for g, h, s in zip(gs, hs, ss):
            g.decode(stream=s)
            h.prefill(stream=s)
    torch.cuda.synchronize()
    for g, h in zip(gs, hs):
        g.check(what="decode")
        h.check(what="prefill")


def test_one_workspace_many_shapes(kvq):
    """Calls of other shapes in turn over one workspace that fits the largest."""
    shapes = [([2000], 32, 8, 128, [5]), ([40] * 20, 8, 2, 64, [1] * 20), ([600, 700], 16, 16, 64, [200, 9])]
    gs = [OnGpu(kvq, f4.Batch(50 + i, lens, hq, hkv, dh), c) for i, (lens, hq, hkv, dh, c) in enumerate(shapes)]
    ws = max((g.ws for g in gs), key=lambda w: w.numel())
    one = [OnGpu(kvq, f4.Batch(60 + i, lens, hq, hkv, dh), [1] * len(lens)) for i, (lens, hq, hkv, dh, _) in enumerate(shapes)]
    for g in gs + one:
        g.ws = ws
    for _ in range(3):
        for g, o in zip(gs, one):
            g.prefill()
            g.check(what="prefill")
            o.decode()
            o.check(what="decode")


def test_offsets_past_32_bits(kvq):
    """A pool of more than 2^32 bytes: pages at its end are written, read and attended to."""
    hq, hkv, dh = 8, 8, 128
    nb = (1 << 32) // (hkv * 9 * dh) + 40
    b = f4.Batch(70, [40], hq, hkv, dh)
    table = (nb - 1 - np.arange(3, dtype=np.int32)).reshape(1, 3)
    pos = np.arange(40)
    slots = table[0, pos // 16].astype(np.int64) * 16 + pos % 16
    kc = torch.empty((nb, hkv, 9 * dh), dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    kvq.kvq_fp4_write(dev(b.k), dev(b.v), dev(slots), kc, vc, dev(b.ks), dev(b.vs), b.gran)
    small = np.array([[2, 1, 0]], np.int32)
    K, V = f4.new_cache(3, hkv, dh), f4.new_cache(3, hkv, dh)
    f4.write(b.k, small[0, pos // 16] * 16 + pos % 16, K, b.ks)
    f4.write(b.v, small[0, pos // 16] * 16 + pos % 16, V, b.vs)
    ko = torch.zeros((40, hkv, dh), dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    cu = np.array([0, 40], np.int32)
    kvq.kvq_fp4_read(kc, vc, dev(table), None, dev(cu), dev(b.ks), dev(b.vs), b.gran, ko, vo)
    assert np.array_equal(bits(ko), f4.read(K, b.ks, small, None, cu, 40))
    assert np.array_equal(bits(vo), f4.read(V, b.vs, small, None, cu, 40))
    q, qcu = b.queries([40])
    ws, out = workspace(kvq, 1, hq, hkv, dh), torch.zeros((40, hq, dh), dtype=torch.bfloat16, device="cuda")
    want, tol = f4.attention(q, K, V, b.ks, b.vs, small, np.array([40]), qcu, 0, 0)
    sl = dev(np.array([40], np.int32))
    kvq.kvq_fp4_prefill_attn(dev(q), dev(qcu), 40, kc, vc, dev(table), sl, dev(b.ks), dev(b.vs), b.gran, 0, 0, ws, out)
    f4.check(bits(out), want, tol, "prefill")
    kvq.kvq_fp4_decode_attn(dev(q[39:]), kc, vc, dev(table), sl, dev(b.ks), dev(b.vs), b.gran, 0, 0, ws, out[:1])
    f4.check(bits(out)[:1], want[39:], tol[39:], "decode")


def test_refusals_reach_no_kernel(kvq):
    """What only real CUDA tensors can show: types, shapes, layouts, workspaces."""
    b = f4.Batch(80, [40], 8, 2, 64)
    g = OnGpu(kvq, b, [1])

    def refused(status, call):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert e.value.status == status, str(e.value)

    ws = g.ws
    g.ws = ws[:kvq.KVQ_WS_COUNTER_BYTES - 16]
    refused(kvq.KVQ_ERR_WORKSPACE, g.decode)
    refused(kvq.KVQ_ERR_WORKSPACE, g.prefill)
    g.ws = ws[16:]
    refused(kvq.KVQ_ERR_ALIGN, g.decode)
    g.ws = ws
    refused(kvq.KVQ_ERR_ARG, lambda: g.decode(window=-1))
    refused(kvq.KVQ_ERR_ARG, lambda: g.decode(sinks=-1))
    g.sl = g.sl.long()
    refused(kvq.KVQ_ERR_ARG, g.decode)
    g.sl = dev(b.lens)
    g.bt = g.bt.t()
    refused(kvq.KVQ_ERR_SHAPE, g.decode)
    g.bt = dev(b.table).cpu()
    refused(kvq.KVQ_ERR_ARG, g.decode)
    torch.cuda.synchronize()
    assert bool((g.out == 7).all())
