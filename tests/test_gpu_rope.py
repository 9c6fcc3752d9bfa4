"""kvq_rope_write against the formula in 64 bits, and against kvq_write where it only writes."""
import pytest
import torch

import step_testlib as lib
from step_testlib import BF16, BS, E4M3, E5M2, PER_HEAD, PER_TENSOR, PER_TOKEN_HEAD

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_paged_gb300 as m
    return m


class Case:
    def __init__(self, kvq, N, hq, hkv, dh, fmt, gran=PER_HEAD, axes=1, pairs=None, interleaved=False, norm=(True, True), far=4096,
                 seed=0, gap=0, skip=True):
        g = torch.Generator().manual_seed(seed)
        self.kvq, self.fmt, self.gran, self.inter, self.N, self.hkv, self.dh = kvq, fmt, gran, interleaved, N, hkv, dh
        pairs = dh // 2 if pairs is None else pairs
        w = (hq + 2 * hkv) * dh + gap
        self.qkv = torch.randn(N, w, generator=g).to(torch.bfloat16).cuda()
        cut = self.qkv[:, :(hq + 2 * hkv) * dh].split((hq * dh, hkv * dh, hkv * dh), 1)
        self.q, self.k, self.v = (t.unflatten(1, (-1, dh)) for t in cut)
        self.pos = torch.randint(-far, far + 1, (axes, N), generator=g, dtype=torch.int64).to(torch.int32).cuda()
        self.freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))
        self.axis = (torch.arange(pairs) % axes).to(torch.uint8).cuda() if axes > 1 else None
        self.wq, self.wk = ((torch.rand(dh, generator=g) + 0.5).to(torch.bfloat16).cuda() if n else None for n in norm)
        blocks = N // BS + 3
        perm = torch.randperm(blocks * BS, generator=g)[:N]
        if skip:
            perm[::7] = -1
        self.slots = perm.cuda()
        self.blocks = blocks
        dt = torch.bfloat16 if fmt == BF16 else torch.uint8
        self.caches = [torch.full((blocks, hkv, BS, dh), 3, dtype=dt).cuda() for _ in range(2)]
        if gran == PER_TOKEN_HEAD:
            self.scales = [torch.full((blocks, hkv, BS), -1.0).cuda() for _ in range(2)]
        else:
            self.scales = [(torch.rand(hkv if gran == PER_HEAD else 1, generator=g) + 3.0).cuda() / lib.TOP.get(fmt, 1.0) for _ in range(2)]
        self.out = torch.full((N, hq, dh), 9.0, dtype=torch.bfloat16).cuda()
        self.st = torch.zeros(1, dtype=torch.int32).cuda()

    def call(self, **kw):
        a = dict(q=self.q, k=self.k, v=self.v, positions=self.pos, axis=self.axis, q_weight=self.wq,
                 k_weight=self.wk, eps=EPS, interleaved=self.inter, slot_mapping=self.slots, k_cache=self.caches[0], v_cache=self.caches[1],
                 k_scale=self.scales[0], v_scale=self.scales[1], scale_granularity=self.gran, fmt=self.fmt, q_out=self.out,
                 dev_status=self.st) | kw
        if "turns" not in a:
            a["turns"] = self.kvq.rope_turns(self.freq)
        self.kvq.kvq_rope_write(**a)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.st.item()) == status
        # binary32 on the way: a norm's 2^-20 relative, a rotation's 2^-20 of its pair
        zq, size = lib.rotated(self.q, self.wq, EPS, self.pos, self.freq, self.axis, self.inter)
        assert bool(((self.out.double() - zq).abs() <= 2.0 ** -8 * zq.abs() + 2.0 ** -18 * size + 1e-38).all())
        zk, size = lib.rotated(self.k, self.wk, EPS, self.pos, self.freq, self.axis, self.inter)
        written = torch.zeros(self.blocks * BS, dtype=torch.bool, device="cuda")
        good = (self.slots >= 0) & (self.slots < self.blocks * BS)
        s, at = self.slots[good], good.nonzero()[:, 0]
        written[s] = True
        for i, (z, err) in enumerate(((zk, size), (self.v.double(), self.v.double() * 0))):
            cache, scale = self.caches[i], self.scales[i]
            got, z, err = lib.decode(cache, self.fmt)[s // BS, :, s % BS], z[at], err[at]
            if self.fmt != BF16:
                if self.gran == PER_TOKEN_HEAD:
                    sc = scale[s // BS, :, s % BS].double()[..., None]
                    top = z.abs().amax(-1, keepdim=True)
                    assert bool(((sc * lib.TOP[self.fmt] - top).abs() <= 2.0 ** -18 * err.amax(-1, keepdim=True) + 2.0 ** -22 * top).all())
                else:
                    sc = scale.double().view(1, -1, 1)
                z, err = (z / sc), err / sc
                z = z.clamp(-lib.TOP[self.fmt], lib.TOP[self.fmt])
            tol = lib.HALF[self.fmt] * z.abs() + lib.LEAST[self.fmt] + 2.0 ** -17 * err + 2.0 ** -22 * z.abs()
            assert bool(((got - z).abs() <= tol).all())
            # nothing else is written
            rest = cache.permute(0, 2, 1, 3).reshape(-1, self.hkv, self.dh)[~written]
            assert bool((rest == 3).all())


SHAPES = [(1, 1, 1, 64), (3, 8, 2, 64), (33, 32, 8, 128), (257, 28, 4, 128), (130, 6, 2, 64), (700, 5, 5, 128), (2000, 7, 1, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", [E4M3, E5M2, BF16])
def test_shapes(kvq, shape, fmt):
    c = Case(kvq, *shape, fmt, gap=8 * (shape[0] % 3), seed=shape[0])
    c.call()
    c.check()


@pytest.mark.parametrize("pairs,interleaved", [(0, False), (8, False), (8, True), (24, False), (24, True), (32, True), (16, False),
                                               (64, True), (40, False)])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("norm", [(True, True), (False, False), (True, False), (False, True)])
def test_rotations(kvq, pairs, interleaved, axes, norm):
    dh = 128 if pairs > 32 else 64
    c = Case(kvq, 37, 6, 2, dh, E4M3, axes=axes, pairs=pairs, interleaved=interleaved, norm=norm, seed=pairs)
    c.call()
    c.check()


@pytest.mark.parametrize("gran", [PER_TENSOR, PER_HEAD, PER_TOKEN_HEAD])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dh", [64, 128])
def test_granularities(kvq, gran, fmt, dh):
    c = Case(kvq, 90, 8, 4, dh, fmt, gran, seed=gran)
    c.call()
    c.check()


@pytest.mark.parametrize("far", [1, 131072, 2 ** 31 - 1])
def test_far_positions(kvq, far):
    """Angles are as exact far away as near: turns are multiplied modulo 2^64.  (A turn is off by 2^-53 of itself, as
    the plain form's angles are: at 2^31 positions of 1 radian 2^-22.)"""
    c = Case(kvq, 64, 4, 2, 128, BF16, far=far, seed=5)
    c.call()
    c.check()


@pytest.mark.parametrize("gran", [PER_TENSOR, PER_HEAD, PER_TOKEN_HEAD])
@pytest.mark.parametrize("fmt", [E4M3, E5M2, BF16])
@pytest.mark.parametrize("dh", [64, 128])
def test_without_rotation_it_writes_as_kvq_write(kvq, gran, fmt, dh):
    """The same codes, scales and bits, NaN, infinities, zeros and all magnitudes among them."""
    if fmt == BF16 and gran == PER_TOKEN_HEAD:
        pytest.skip("no scales")
    c = Case(kvq, 300, 3, 3, dh, fmt, gran, pairs=0, norm=(False, False), seed=2)
    bits = torch.randint(0, 65536, (300, c.qkv.shape[1]), generator=torch.Generator().manual_seed(9)).to(torch.int32)
    c.qkv.copy_(bits.to(torch.int16).view(torch.bfloat16).cuda().view_as(c.qkv))
    c.call()
    want = [x.clone().fill_(3) for x in c.caches]
    scales = [x.clone() for x in c.scales]
    if gran == PER_TOKEN_HEAD:
        scales = [torch.full_like(x, -1.0) for x in scales]
        kvq.kvq_write_token_head(c.k, c.v, c.slots, *want, *scales, fmt)
    else:
        kvq.kvq_write(c.k, c.v, c.slots, *want, *scales, gran, fmt)
    torch.cuda.synchronize()
    for got, w in zip(c.caches, want):
        if fmt == BF16:
            nan = w.isnan()
            assert bool(((got.view(torch.int16) == w.view(torch.int16)) | nan).all()) and torch.equal(got.isnan(), nan)
        else:
            nan = w.view(lib.F8[fmt]).float().isnan()
            assert bool(((got == w) | nan).all()) and torch.equal(got.view(lib.F8[fmt]).float().isnan(), nan)
    for got, w in zip(c.scales, scales):
        assert torch.equal(got, w)
    assert bool(((c.out == c.q) | (c.out.isnan() & c.q.isnan())).all())


def test_quotients_of_normed_rows(kvq):
    """Codes of z / s for z with 24 significant bits: those of the exact quotient or, where that lies within the
    norm's 2^-20 of a border, the next ones."""
    c = Case(kvq, 4096, 1, 2, 128, E4M3, PER_HEAD, pairs=0, norm=(False, True), skip=False, seed=3)
    c.call()
    torch.cuda.synchronize()
    z, _ = lib.rotated(c.k, c.wk, EPS, c.pos, c.freq, None, False)
    q = z / c.scales[0].double().view(1, -1, 1)
    lo, hi = (lib.decode(lib.encode((q * (1 + e)).float(), E4M3), E4M3) for e in (-2.0 ** -20, 2.0 ** -20))
    got = lib.decode(c.caches[0], E4M3)[c.slots // BS, :, c.slots % BS]
    assert bool(((got == lo) | (got == hi)).all())


def test_in_place_and_strides(kvq):
    a, b = (Case(kvq, 77, 8, 2, 128, E4M3, seed=4, gap=16) for _ in range(2))
    a.call()
    b.call(q_out=b.q)
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.q) and torch.equal(a.caches[0], b.caches[0])
    assert torch.equal(a.qkv[:, -16:], b.qkv[:, -16:]) and torch.equal(a.k, b.k)  # only q's columns changed


def test_bad_slots_are_reported(kvq):
    c = Case(kvq, 40, 4, 2, 64, E4M3, seed=6)
    c.slots[3] = c.blocks * BS
    c.slots[5] = 2 ** 40
    c.call()
    c.check(status=kvq.KVQ_DEV_BAD_SLOT)


def test_nan_stays_in_its_row(kvq):
    c = Case(kvq, 50, 4, 2, 128, E4M3, seed=7, skip=False)
    c.qkv[10, 5] = float("nan")          # q head 0
    c.qkv[11, 4 * 128 + 3] = float("inf")  # k head 0
    ref = Case(kvq, 50, 4, 2, 128, E4M3, seed=7, skip=False)
    c.call()
    ref.call()
    torch.cuda.synchronize()
    assert bool(c.out[10, 0].isnan().all())
    same = torch.ones(50, 4, dtype=torch.bool, device="cuda")
    same[10, 0] = False
    assert torch.equal(c.out[same], ref.out[same])
    s = c.slots
    got, want = (x.caches[0][s // BS, :, s % BS] for x in (c, ref))
    same = torch.ones(50, 2, dtype=torch.bool, device="cuda")
    same[11, 0] = False
    assert torch.equal(got[same], want[same])


def test_no_tokens_and_graph_and_stream(kvq):
    c = Case(kvq, 0, 4, 2, 64, E4M3)
    c.call()
    a, b = (Case(kvq, 60, 8, 2, 64, E5M2, seed=8) for _ in range(2))
    a.call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    turns = kvq.rope_turns(b.freq)
    with torch.cuda.graph(graph, stream=s):
        b.call(turns=turns)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.caches[0], b.caches[0])
    b.out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    b.call(turns=turns, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out)
