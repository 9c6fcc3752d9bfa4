"""The operators of a serving step together, as they are used: drafts written, attended, the accepted path
kept and pages given back; beams forked and gone on with; the same in a graph."""
import random

import pytest
import torch

import step_testlib as lib
from step_testlib import BF16, BS, E4M3, E5M2, PER_HEAD, PER_TOKEN_HEAD

pytestmark = pytest.mark.gpu
HQ, HKV = 8, 2


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_paged_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Sequences over pages of a pool, in two layers' caches, and what every token's rows hold."""

    def __init__(self, kvq, B, dh, fmt, gran, blocks, seed):
        self.kvq, self.dh, self.fmt, self.gran, self.blocks = kvq, dh, fmt, gran, blocks
        self.rng, self.g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.mb = 24
        self.pool = kvq.new_page_pool(blocks)
        self.bt = torch.full((B, self.mb), -1, dtype=torch.int32, device="cuda")
        self.lens = i32([0] * B)
        dt = torch.bfloat16 if fmt == BF16 else torch.uint8
        self.layers = [[torch.full((blocks, HKV, BS, dh), 0x7F, dtype=torch.uint8).to(dt).cuda() for _ in range(2)] for _ in range(2)]
        n = (blocks, HKV, BS) if gran == PER_TOKEN_HEAD else (HKV,)
        self.scales = [[torch.full(n, 0.02, device="cuda") for _ in range(2)] for _ in range(2)]
        self.ws = kvq.new_tree_workspace(HQ, HKV, dh)
        self.turns = kvq.rope_turns([10000.0 ** (-i / 32) for i in range(dh // 2)])
        self.weight = (torch.rand(dh, generator=self.g) + 0.5).to(torch.bfloat16).cuda()
        self.st = i32([0])
        self.rows = [[] for _ in range(B)]  # of each token, every cache's

    def caches(self):
        flat = [c for layer in self.layers for c in layer]
        return flat + ([s for layer in self.scales for s in layer] if self.gran == PER_TOKEN_HEAD else [])

    def gather(self, b, n):
        """Every cache's rows of sequence b's first n tokens."""
        t = torch.arange(n, device="cuda")
        blk = self.bt[b][t // BS].long()
        assert n == 0 or int(blk.min()) >= 0
        return [[c.view(torch.uint8).unflatten(-1, (BS, 4))[blk, :, t % BS] if c.dim() == 3 else c[blk, :, t % BS] for c in self.caches()]][0]

    def write(self, new_lens, positions, slots):
        """Both layers' rows of new tokens; the queries."""
        N = slots.numel()
        out = []
        for (kc, vc), (ks, vs) in zip(self.layers, self.scales):
            qkv = torch.randn(N, (HQ + 2 * HKV) * self.dh, generator=self.g).to(torch.bfloat16).cuda()
            q, k, v = (x.unflatten(1, (-1, self.dh)) for x in qkv.split([HQ * self.dh, HKV * self.dh, HKV * self.dh], 1))
            o = torch.empty(N, HQ, self.dh, dtype=torch.bfloat16, device="cuda")
            self.kvq.kvq_rope_write(q, k, v, positions, self.turns, None, self.weight, self.weight, 1e-6, False, slots, kc, vc, ks, vs,
                                    self.gran, self.fmt, o, self.st)
            out.append(o)
        return out

    def slots(self, b, first, n):
        t = torch.arange(first, first + n, device="cuda")
        return self.bt[b][t // BS].long() * BS + t % BS

    def attend(self, q, layer, cu, parents):
        kc, vc = self.layers[layer]
        out = torch.full_like(q, 5.0)
        self.kvq.kvq_tree_attn(q, cu, parents, kc, vc, self.bt, self.lens, *self.scales[layer], self.gran, self.fmt, 0, self.ws, out, self.st)
        return out

    def check_attention(self, q, out, layer, trees):
        r = lib.TreeBatch.__new__(lib.TreeBatch)
        r.lens, r.nodes, r.parents = self.lens.tolist(), [len(t) for t in trees], trees
        r.hq, r.hkv, r.dh, r.fmt, r.gran, r.window, r.qs, r.q, r.dev, r.nb, r.bt = HQ, HKV, self.dh, self.fmt, self.gran, 0, None, q, "cuda", self.blocks, self.bt
        r.cu = torch.tensor([0] + torch.tensor(r.nodes).cumsum(0).tolist())
        for name, c, s in zip("KV", self.layers[layer], self.scales[layer]):
            w = 1.0 if self.fmt == BF16 else s.double()[..., None] if self.gran == PER_TOKEN_HEAD else s.double().view(1, -1, 1, 1)
            setattr(r, name, lib.decode(c, self.fmt) * w)
        ref, bound = r.reference()
        assert bool(((out.double() - ref).abs() <= bound).all())

    def step(self, graph=False):
        """A step of speculative decoding: a tree of drafts for each sequence, of which a path is kept."""
        B = len(self.rows)
        counts = [self.rng.choice((0, 1, 3, 9, 17, 30)) for _ in range(B)]
        trees = [lib.random_parents(n, self.g) for n in counts]
        before = self.lens.tolist()
        # (a sequence near its table's end stays as it is)
        trees = [t if L + len(t) <= self.mb * BS else [] for t, L in zip(trees, before)]
        counts = [len(t) for t in trees]
        want = i32([L + n for L, n in zip(before, counts)])
        old = self.lens.clone()
        self.kvq.kvq_pages_alloc(self.pool, self.bt, old, want, self.st)
        self.lens = want
        torch.cuda.synchronize()
        assert int(self.st) == 0
        N = sum(counts)
        cu = i32([0] + torch.tensor(counts).cumsum(0).tolist())
        parents = i32([p for t in trees for p in t] + [0] * (N == 0))[:N]
        depth = [[len(lib.way_up(t, j)) - 1 for j in range(len(t))] for t in trees]
        positions = i32([L + d for L, ds in zip(before, depth) for d in ds] + [0])[:N]
        slots = torch.cat([self.slots(b, L, n) for b, (L, n) in enumerate(zip(before, counts))])
        queries = self.write(want, positions, slots)
        outs = [self.attend(q, i, cu, parents) for i, q in enumerate(queries)]
        if N:
            for i, (q, o) in enumerate(zip(queries, outs)):
                self.check_attention(q, o, i, trees)
        # a path from a random node up is what was accepted
        paths = []
        for t in trees:
            way = sorted(lib.way_up(t, self.rng.randrange(len(t)))) if t else []
            paths.append(way[:self.rng.randint(0, len(way))])
        most = max(map(len, paths)) + 1
        accepted = i32([w + [7] * (most - len(w)) for w in paths])
        taken, new = i32([len(w) for w in paths]), torch.zeros_like(self.lens)
        drafted = [self.gather(b, L + n) for b, (L, n) in enumerate(zip(before, counts))]
        self.kvq.kvq_tree_commit(self.caches(), cu, self.bt, self.lens, accepted, taken, new, self.st)
        self.kvq.kvq_pages_free(self.pool, self.bt, self.lens, new, self.st)
        self.lens = new
        torch.cuda.synchronize()
        assert int(self.st) == 0 and new.tolist() == [L + len(w) for L, w in zip(before, paths)]
        for b, (L, w) in enumerate(zip(before, paths)):
            keep = torch.tensor(list(range(L)) + [L + j for j in w], dtype=torch.long, device="cuda")
            for was, now in zip(drafted[b], self.gather(b, L + len(w))):
                assert torch.equal(was[keep].view(torch.uint8), now.view(torch.uint8))
        self.check_pool()

    def check_pool(self):
        held = [0] * self.blocks
        pages = [-(-n // BS) for n in self.lens.tolist()]
        for row, n in zip(self.bt.tolist(), pages):
            assert all(x >= 0 for x in row[:n]) and all(x == -1 for x in row[n:])
            for x in row[:n]:
                held[x] += 1
        p = lib.Pool(self.blocks)
        p.refs = held
        assert self.pool.tolist() == [w for w in p.words()]

    def fork(self, parents):
        """The sequences go on from `parents`."""
        B = len(parents)
        bt, lens, copies = torch.full_like(self.bt[:1], -1).repeat(B, 1), i32([0] * B), i32([[-1, -1]] * B)
        was = [self.gather(s, n) for s, n in enumerate(self.lens.tolist())]
        self.kvq.kvq_pages_fork(self.pool, self.bt, self.lens, i32(parents), bt, lens, copies, self.st)
        self.kvq.kvq_copy_pages(self.caches(), copies, self.st)
        self.kvq.kvq_pages_free(self.pool, self.bt, self.lens, torch.zeros_like(self.lens), self.st)
        torch.cuda.synchronize()
        assert int(self.st) == 0 and lens.tolist() == [self.lens.tolist()[s] for s in parents]
        self.bt, self.lens, self.rows = bt, lens, [[] for _ in parents]
        for b, s in enumerate(parents):
            for x, y in zip(was[s], self.gather(b, int(lens[b]))):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        self.check_pool()


@pytest.mark.parametrize("fmt,gran,dh", [(E4M3, PER_HEAD, 128), (E5M2, PER_TOKEN_HEAD, 64), (BF16, PER_HEAD, 128)])
def test_serving_loop(kvq, fmt, gran, dh):
    """Steps of drafts and commits, beams that fork between them: pages that are shared are never written."""
    s = Server(kvq, 5, dh, fmt, gran, 200, seed=dh + fmt)
    for i in range(9):
        s.step()
        if i in (3, 6):
            s.fork([s.rng.randrange(len(s.rows)) for _ in range(6)])


def test_captured_step(kvq):
    """Write, attention, commit and free in one graph, replayed over restored caches: the eager run's bits."""
    b = lib.TreeBatch([(300, 20), (77, 7), (1000, 40)], HQ, HKV, 128, E4M3, seed=3)
    N, new, st = b.q.shape[0], torch.zeros(3, dtype=torch.int32, device="cuda"), i32([0])
    qkv = torch.randn(N, (HQ + 2 * HKV) * 128, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    q, k, v = (x.unflatten(1, (-1, 128)) for x in qkv.split([HQ * 128, HKV * 128, HKV * 128], 1))
    slots = torch.cat([b.bt[i].long()[torch.arange(L - n, L) // BS] * BS + torch.arange(L - n, L, device="cuda") % BS
                       for i, (L, n) in enumerate(zip(b.lens, b.nodes))])
    turns, pos = kvq.rope_turns([0.5 ** i for i in range(64)]), torch.arange(N, dtype=torch.int32, device="cuda")
    paths = [lib.way_up(b.parents[i], b.nodes[i] - 1)[::-1] for i in range(3)]
    most = max(map(len, paths))
    accepted, taken = i32([sorted(w) + [0] * (most - len(w)) for w in paths]), i32([len(w) for w in paths])
    pool = kvq.new_page_pool(b.nb)
    held = torch.bincount(b.bt[b.bt >= 0].long(), minlength=b.nb).to(torch.int32)
    pool[4:4 + b.nb] = held
    pool[1] = int((held == 0).sum())
    free = (held == 0).cpu().tolist()
    words = [sum(1 << j for j in range(32) if 32 * i + j < b.nb and free[32 * i + j]) for i in range((b.nb + 31) // 32)]
    pool[4 + b.nb:] = i32([w - (1 << 32) if w >> 31 else w for w in words])
    state = [b.kc, b.vc, b.bt, pool, new]
    saved = [t.clone() for t in state]
    rot, out, ws = torch.empty_like(b.q), torch.empty_like(b.q), kvq.new_tree_workspace(HQ, HKV, 128)

    def run():
        kvq.kvq_rope_write(q, k, v, pos, turns, None, None, None, 0.0, False, slots, b.kc, b.vc, b.ks, b.vs, b.gran, E4M3, rot, st)
        kvq.kvq_tree_attn(rot, b.cu_d, b.par, b.kc, b.vc, b.bt, b.sl, b.ks, b.vs, b.gran, E4M3, 0, ws, out, st)
        kvq.kvq_tree_commit([b.kc, b.vc], b.cu_d, b.bt, b.sl, accepted, taken, new, st)
        kvq.kvq_pages_free(pool, b.bt, b.sl, new, st)

    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in state + [rot, out]]
    assert int(st) == 0 and bool(out.isfinite().all())
    for t, s in zip(state, saved):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t, s in zip(state, saved):
            t.copy_(s)
        rot.zero_(), out.zero_(), ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert int(st) == 0
        for t, w in zip(state + [rot, out], want):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))


def test_two_streams_at_once(kvq):
    """Two batches' attentions at the same time, a workspace each: the bits of one after the other."""
    bs = [lib.TreeBatch([(3000, 30), (500, 9)], HQ, HKV, 128, E4M3, seed=s) for s in (1, 2)]
    gs = [lib.OnGpu(kvq, b) for b in bs]
    want = [g.call().clone() for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(20):
        for g, s in zip(gs, streams):
            with torch.cuda.stream(s):
                g.call()
    torch.cuda.synchronize()
    for g, w in zip(gs, want):
        assert torch.equal(g.out.view(torch.uint8), w.view(torch.uint8)) and int(g.st) == 0


def test_caches_past_32_bits(kvq):
    """The same step on pages at the end of caches of 4.4 GB: the small caches' bits."""
    far, small, hkv, dh = 270000 - 40, 40, 8, 128
    N, g = 30, torch.Generator().manual_seed(5)
    qkv = torch.randn(N, (16 + 2 * hkv) * dh, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv.split([16 * dh, hkv * dh, hkv * dh], 1))
    fill = torch.randint(0, 120, (2, small, hkv, BS, dh), generator=g, dtype=torch.uint8).cuda()
    scale, turns, pos = torch.full((hkv,), 0.02, device="cuda"), kvq.rope_turns([0.3 ** i for i in range(64)]), torch.arange(N, dtype=torch.int32, device="cuda")
    parents, accepted = i32([-1] + [i // 2 for i in range(N - 1)]), i32([[0, 2, 5, 12]])
    ws, cu = kvq.new_tree_workspace(16, hkv, dh), i32([0, N])
    results = []
    for at in (0, far):
        caches = [torch.empty(at + small, hkv, BS, dh, dtype=torch.uint8, device="cuda") for _ in range(2)]
        for c, f in zip(caches, fill):
            c[at:] = f
        bt = (torch.arange(30, dtype=torch.int32, device="cuda").flip(0) + at)[None].contiguous()
        lens, new, st = i32([450 + N]), i32([0]), i32([0])
        t = torch.arange(450, 450 + N, device="cuda")
        slots = bt[0][t // BS].long() * BS + t % BS
        rot, out = torch.empty_like(q).contiguous(), torch.empty(N, 16, dh, dtype=torch.bfloat16, device="cuda")
        kvq.kvq_rope_write(q, k, v, pos, turns, None, None, None, 0.0, False, slots, *caches, scale, scale, PER_HEAD, E4M3, rot, st)
        kvq.kvq_tree_attn(rot, cu, parents, *caches, bt, lens, scale, scale, PER_HEAD, E4M3, 0, ws, out, st)
        kvq.kvq_tree_commit(caches, cu, bt, lens, accepted, i32([4]), new, st)
        kvq.kvq_copy_pages(caches, i32([[at + 3, at + 39], [at + 29, at + 35]]), st)
        torch.cuda.synchronize()
        assert int(st) == 0 and int(new) == 454
        results.append([rot, out] + [c[at:].clone() for c in caches])
        del caches
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_batches_without_a_tree(kvq):
    """Sequences of no nodes, empty ones among them: nothing is read of them and no row is written."""
    for lens in ([0, 20, 0], [0], [300] * 500):
        B = len(lens)
        kc = torch.full((4, HKV, BS, 64), 0x7F, dtype=torch.uint8, device="cuda")
        q, st = torch.randn(3, HQ, 64, device="cuda").to(torch.bfloat16), i32([0])
        out = torch.full_like(q, 7.0)
        bt = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
        kvq.kvq_tree_attn(q, i32([0] * (B + 1)), None, kc, kc.clone(), bt, i32(lens), *[torch.ones(1, device="cuda")] * 2, 0, E4M3, 0,
                          kvq.new_tree_workspace(HQ, HKV, 64), out, st)
        torch.cuda.synchronize()
        assert int(st) == 0 and bool((out == 7.0).all())


def test_another_stream_by_argument(kvq):
    """A call on a stream that is not the current one is ordered with that stream's work."""
    b = lib.TreeBatch([(2000, 20)], HQ, HKV, 128, E4M3, seed=6)
    g = lib.OnGpu(kvq, b)
    want = g.call().clone()
    s, q = torch.cuda.Stream(), b.q.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late = torch.zeros_like(q)
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
    g.out.fill_(7.0)
    torch.cuda.current_stream().synchronize()
    g.call(q=late, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(g.out.view(torch.uint8), want.view(torch.uint8)) and int(g.st) == 0
