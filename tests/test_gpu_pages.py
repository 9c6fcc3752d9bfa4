"""Rows and pages moved, and the pool: bit for bit against plain Python."""
import random

import pytest
import torch

import step_testlib as lib
from step_testlib import BS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_paged_gb300 as m
    return m


def make_caches(blocks, hkv, dh, kinds, seed=0):
    g = torch.Generator().manual_seed(seed)
    made = []
    for kind in kinds:
        shape = {"fp8": (blocks, hkv, BS, dh), "bf16": (blocks, hkv, BS, 2 * dh), "scale": (blocks, hkv, BS * 4), "fp4": (blocks, hkv, 9 * dh)}[kind]
        c = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()
        made.append({"bf16": lambda t: t.view(torch.bfloat16), "scale": lambda t: t.view(torch.float32)}.get(kind, lambda t: t)(c))
    return made


def rows_view(c):
    """Byte views [blocks][hkv][16][row bytes] of a cache's rows."""
    b = c.view(torch.uint8)
    if c.dim() == 3 and c.dtype == torch.float32:
        return [b.view(*c.shape[:2], BS, 4)]
    if c.dim() == 3:
        dh = c.shape[2] // 9
        return [b[..., :8 * dh].unflatten(2, (BS, dh // 2)), b[..., 8 * dh:].unflatten(2, (BS, dh // 16))]
    return [b]


def commit_plain(caches, bt, moves):
    """moves: per sequence (tokens before the tree, path)."""
    for c in caches:
        for view in rows_view(c):
            new = view.clone()
            for b, (P, path) in enumerate(moves):
                for i, j in enumerate(path):
                    s, d = P + j, P + i
                    new[int(bt[b][d // BS]), :, d % BS] = view[int(bt[b][s // BS]), :, s % BS]
            view.copy_(new)


def run_commit(kvq, seqs, paths, kinds, hkv, dh, seed=0, **kw):
    """seqs: (tokens, nodes); paths: accepted nodes of each."""
    pages = [-(-n // BS) for n, _ in seqs]
    nb = sum(pages) + 2
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).tolist()
    bt = torch.full((len(seqs), max(pages) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    caches, want = (make_caches(nb, hkv, dh, kinds, seed) for _ in range(2))
    width = max(1, max(len(p) for p in paths))
    path = torch.tensor([p + [-5] * (width - len(p)) for p in paths], dtype=torch.int32).cuda()
    taken = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
    lens = torch.tensor([n for n, _ in seqs], dtype=torch.int32).cuda()
    cu = torch.tensor([0] + torch.tensor([m for _, m in seqs]).cumsum(0).tolist(), dtype=torch.int32).cuda()
    out, st = torch.full_like(lens, -9), torch.zeros(1, dtype=torch.int32).cuda()
    args = dict(caches=caches, cu_q_lens=cu, block_tables=bt.cuda(), seq_lens=lens, accepted=path, num_accepted=taken, new_lens=out,
                dev_status=st) | kw
    kvq.kvq_tree_commit(**args)
    torch.cuda.synchronize()
    return caches, want, bt, out.tolist(), int(st.item())


KINDS = (["fp8"], ["bf16"], ["fp4"], ["fp8", "scale", "bf16", "fp4", "scale"])


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("hkv,dh", [(1, 64), (2, 128), (8, 128), (5, 64)])
def test_commit(kvq, kinds, hkv, dh):
    rng = random.Random(hkv * dh)
    seqs = [(rng.randint(n, n + 70), n) for n in (1, 2, 9, 40, 17, 64, 200)]
    paths = [sorted(rng.sample(range(n), rng.randint(0, n))) for _, n in seqs]
    paths[3] = list(range(40))  # everything stays
    paths[5] = list(range(1, 64))  # everything moves by one: each row is another's place
    paths[6] = list(range(0, 200, 2))  # more than a warp holds at once
    caches, want, bt, lens, st = run_commit(kvq, seqs, paths, kinds, hkv, dh, seed=1)
    commit_plain(want, bt, [(L - n, p) for (L, n), p in zip(seqs, paths)])
    assert st == 0 and lens == [L - n + len(p) for (L, n), p in zip(seqs, paths)]
    for got, w in zip(caches, want):
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))


def test_commit_many_caches(kvq):
    """More caches than one launch takes."""
    seqs, paths = [(40, 9), (21, 5)], [[0, 3, 7], [2]]
    caches, want, bt, lens, st = run_commit(kvq, seqs, paths, ["fp8", "scale"] * 150, 2, 64)
    commit_plain(want, bt, [(L - n, p) for (L, n), p in zip(seqs, paths)])
    assert st == 0 and lens == [34, 17]
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(caches, want))


def test_commit_what_is_wrong_moves_nothing(kvq):
    seqs = [(50, 10)] * 6
    paths = [[0, 2, 2], [3, 1], [4, 10], [1, 5], [-1, 3], [2, 6]]  # a repeat, a fall, past the tree, good, below, good
    caches, want, bt, lens, st = run_commit(kvq, seqs, paths, ["fp8", "fp4"], 2, 64)
    assert st == kvq.KVQ_DEV_BAD_TREE and lens == [50, 50, 50, 42, 50, 42]
    commit_plain(want, bt, [(40, p if i in (3, 5) else []) for i, p in enumerate(paths)])
    assert all(torch.equal(a, b) for a, b in zip(caches, want))
    taken = torch.tensor([3, 2, 2, 2, -1, 11], dtype=torch.int32).cuda()
    _, _, _, lens, st = run_commit(kvq, seqs, [[0, 1, 2]] + [[1, 5]] * 5, ["fp8"], 2, 64, num_accepted=taken)
    assert st == kvq.KVQ_DEV_BAD_TREE and lens == [43, 42, 42, 42, 50, 50]
    # lengths that do not hold the tree, or that the table does not hold; falling offsets
    sl = torch.tensor([50, 9, -1, 10 ** 6, 50, 50], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 10, 20, 30, 40, 35, 45], dtype=torch.int32).cuda()
    caches, want, bt, lens, st = run_commit(kvq, seqs, [[1, 5]] * 6, ["fp8"], 2, 64, seq_lens=sl, cu_q_lens=cu)
    assert st == kvq.KVQ_DEV_BAD_SEQLEN | kvq.KVQ_DEV_BAD_QLEN and lens == [42, 9, -1, 10 ** 6, 50, 42]


def test_commit_bad_pages(kvq):
    seqs, paths = [(50, 20)], [[3, 4, 15]]  # tokens 33, 34, 45 to 30, 31, 32
    bt = torch.tensor([[1, 2, 0, 99]], dtype=torch.int32)  # tokens 48, 49 lie on no page
    caches, want, _, lens, st = run_commit(kvq, seqs, paths, ["fp8"], 2, 64, block_tables=bt.cuda())
    commit_plain(want, bt, [(30, paths[0])])
    assert st == 0 and lens == [33] and all(torch.equal(a, b) for a, b in zip(caches, want))
    bt[0, 2] = -1
    caches, want, _, lens, st = run_commit(kvq, seqs, paths, ["fp8"], 2, 64, block_tables=bt.cuda())
    assert st == kvq.KVQ_DEV_BAD_BLOCK and lens == [33] and all(torch.equal(a, b) for a, b in zip(caches, want))


def test_commit_empty(kvq):
    t = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    c = make_caches(3, 2, 64, ["fp8"])
    kvq.kvq_tree_commit(c, t(1), t(0, 4), t(0), t(0, 3), t(0), t(0))
    lens = torch.full((2,), 5, dtype=torch.int32).cuda()
    out = t(2)
    kvq.kvq_tree_commit(c, t(3), t(2, 4), lens, t(2, 0), t(2), out)  # paths without places
    torch.cuda.synchronize()
    assert out.tolist() == [5, 5]


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("n", [1, 7, 300])
def test_copy(kvq, kinds, n):
    nb, rng = 2 * n + 5, random.Random(n)
    ids = rng.sample(range(nb), 2 * n)
    pairs = [[ids[2 * i], ids[2 * i + 1]] for i in range(n)]
    got, want = (make_caches(nb, 3, 64, kinds, n) for _ in range(2))
    if n > 1:
        pairs[1] = [-1, ids[3]]
        pairs[2] = [ids[4], -1]
    for c in want:
        for s, d in pairs:
            if s >= 0 and d >= 0:
                c[d] = c[s]
    st = torch.zeros(1, dtype=torch.int32).cuda()
    kvq.kvq_copy_pages(got, torch.tensor(pairs, dtype=torch.int32).cuda(), dev_status=st)
    kvq.kvq_copy_pages(got, torch.zeros(0, 2, dtype=torch.int32).cuda(), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    kvq.kvq_copy_pages(got, torch.tensor([[0, nb], [nb, 1]], dtype=torch.int32).cuda(), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == kvq.KVQ_DEV_BAD_BLOCK
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


class Held:
    """A pool and its tables, on the GPU and in Python."""

    def __init__(self, kvq, blocks, B, mb):
        self.kvq, self.mb, self.plain = kvq, mb, lib.Pool(blocks)
        self.pool = kvq.new_page_pool(blocks)
        self.tables, self.rows = torch.full((B, mb), -1, dtype=torch.int32).cuda(), [[-1] * mb for _ in range(B)]
        self.st = torch.zeros(1, dtype=torch.int32).cuda()

    def t(self, x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def alloc(self, old, new):
        self.kvq.kvq_pages_alloc(self.pool, self.tables, self.t(old), self.t(new), dev_status=self.st)

    def free(self, old, new):
        self.kvq.kvq_pages_free(self.pool, self.tables, self.t(old), self.t(new), dev_status=self.st)

    def same(self, status=0):
        torch.cuda.synchronize()
        assert int(self.st.item()) == status
        self.st.zero_()
        assert self.tables.tolist() == self.rows
        assert self.pool.tolist() == self.plain.words()


@pytest.mark.parametrize("blocks,B,most", [(7, 1, 60), (200, 9, 200), (5000, 64, 700), (200000, 300, 3000), (33, 40, 20), (131073, 4096, 400)])
def test_pool_over_a_serving_loop(kvq, blocks, B, most):
    """Steps of random growth, shrinking and forking; some are refused for want of pages."""
    rng = random.Random(blocks)
    h = Held(kvq, blocks, B, -(-most // BS) + 2)
    lens = [0] * B
    for step in range(5):
        new = [rng.choice((n, 0, rng.randint(0, most), min(most, n + rng.randint(0, 40)))) for n in lens]
        up = [max(a, z) for a, z in zip(lens, new)]
        h.alloc(lens, up)
        if h.plain.alloc(h.rows, lens, up):
            lens = up
            h.same()
        else:
            h.same(kvq.KVQ_DEV_NO_PAGES)
        down = [min(a, z) for a, z in zip(lens, new)]
        h.free(lens, down)
        h.plain.give(h.rows, lens, down)
        lens = down
        h.same()
        parents = [rng.choice((-1, rng.randrange(B), rng.randrange(max(1, B // 8)))) for _ in range(B)]
        out = torch.full((B, h.mb), 77, dtype=torch.int32).cuda()
        out_lens, copies = torch.full((B,), 77, dtype=torch.int32).cuda(), torch.full((B, 2), 77, dtype=torch.int32).cuda()
        kvq.kvq_pages_fork(h.pool, h.tables, h.t(lens), h.t(parents), out, out_lens, copies, dev_status=h.st)
        want = h.plain.fork(h.rows, lens, parents, h.mb)
        if want is None:
            h.same(kvq.KVQ_DEV_NO_PAGES)
            assert bool((out == 77).all() & (out_lens == 77).all() & (copies == 77).all())
            continue
        h.same()
        assert out.tolist() == want[0] and out_lens.tolist() == want[1] and copies.tolist() == want[2]
        # the old tables go, the new ones stay
        h.free(lens, [0] * B)
        h.plain.give(h.rows, lens, [0] * B)
        h.same()
        h.tables, h.rows, lens = out, want[0], want[1]
    h.free(lens, [0] * B)
    torch.cuda.synchronize()
    assert int(h.pool[1]) == blocks


def test_pool_init(kvq):
    for n in (1, 31, 32, 33, 5000):
        pool = torch.full_like(kvq.new_page_pool(n), 123)
        kvq.kvq_pages_init(pool)
        torch.cuda.synchronize()
        assert pool.tolist() == lib.Pool(n).words() == kvq.new_page_pool(n).tolist()


def test_pool_bad_lengths_and_pages(kvq):
    h = Held(kvq, 40, 4, 5)
    h.alloc([0, -1, 0, 0], [33, 16, 81, 80])
    h.plain.alloc(h.rows, [0, 0, 0, 0], [33, 0, 0, 80])
    h.same(kvq.KVQ_DEV_BAD_SEQLEN)
    h.free([33, 0, 0, 80], [0, -3, 0, 1000])
    h.plain.give(h.rows, [33], [0])
    h.same(kvq.KVQ_DEV_BAD_SEQLEN)
    # an entry that is no page, one that nothing holds, and one given back twice
    keep = h.rows[3][0]
    h.tables[0, :4] = h.t([-1, 40, 39, keep])
    h.tables[1, 0] = keep
    h.free([64, 16, 0, 0], [0, 0, 0, 0])
    torch.cuda.synchronize()
    assert int(h.st.item()) == kvq.KVQ_DEV_BAD_BLOCK and bool((h.tables[:2] == -1).all())
    h.plain.refs[keep] = 0
    assert h.pool.tolist() == h.plain.words()


def test_fork_bad_rows(kvq):
    h = Held(kvq, 40, 4, 5)
    lens = [40, 20, 16, 7]
    h.alloc([0] * 4, lens)
    h.plain.alloc(h.rows, [0] * 4, lens)
    h.same()
    h.tables[0, 1] = 39  # held by nothing
    h.tables[1, 1] = 41  # no page, where the last tokens are
    out, out_lens, copies = (torch.zeros(s, dtype=torch.int32).cuda() for s in ((6, 5), (6,), (6, 2)))
    src = h.t([40, 20, 81, 7])
    kvq.kvq_pages_fork(h.pool, h.tables, src, h.t([0, 1, 2, 3, 4, -1]), out, out_lens, copies, dev_status=h.st)
    torch.cuda.synchronize()
    assert int(h.st.item()) == kvq.KVQ_DEV_BAD_SEQLEN | kvq.KVQ_DEV_BAD_BLOCK
    a = h.plain.free()[:2]
    assert out.tolist() == [[h.rows[0][0], -1, a[0], -1, -1], [h.rows[1][0], -1, -1, -1, -1], [-1] * 5, [a[1], -1, -1, -1, -1], [-1] * 5, [-1] * 5]
    assert out_lens.tolist() == [40, 20, 0, 7, 0, 0]
    assert copies.tolist() == [[h.rows[0][2], a[0]], [-1, -1], [-1, -1], [h.rows[3][0], a[1]], [-1, -1], [-1, -1]]
    for i in (h.rows[0][0], h.rows[1][0], *a):
        h.plain.refs[i] += 1
    assert h.pool.tolist() == h.plain.words()


def test_fork_in_a_graph(kvq):
    """Captured and replayed: free, fork, copy, alloc as a step of beams makes them."""
    h = Held(kvq, 200, 8, 6)
    lens = [20 + 3 * i for i in range(8)]
    h.alloc([0] * 8, lens)
    h.plain.alloc(h.rows, [0] * 8, lens)
    h.same()
    caches = make_caches(200, 2, 64, ["fp8", "fp4"])
    out, out_lens, copies, zero = (torch.zeros(s, dtype=torch.int32).cuda() for s in ((8, 6), (8,), (8, 2), (8,)))
    have, src, parents = torch.zeros_like(out_lens), h.t(lens), h.t([0, 0, 1, 5, 5, 5, 7, -1])

    def step():
        kvq.kvq_pages_free(h.pool, out, have, zero, dev_status=h.st)
        kvq.kvq_pages_fork(h.pool, h.tables, src, parents, out, out_lens, copies, dev_status=h.st)
        kvq.kvq_copy_pages(caches, copies, dev_status=h.st)
        have.copy_(out_lens + 9)
        kvq.kvq_pages_alloc(h.pool, out, out_lens, have, dev_status=h.st)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    got = []
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert int(h.st.item()) == 0
        got.append((out.tolist(), h.pool.tolist(), copies.tolist()))
        for s, d in copies.tolist():
            if s >= 0:
                assert all(torch.equal(c[s], c[d]) for c in caches)
    assert got[0] == got[1] == got[2]
