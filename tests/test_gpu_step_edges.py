"""Ordinary calls of the step's operators at the edges of what they take."""
import random

import pytest
import torch

import step_testlib as lib
from test_gpu_pages import commit_plain, kvq, make_caches  # noqa: F401
from test_gpu_rope import Case

pytestmark = pytest.mark.gpu


def test_commit_arrays_side_by_side(kvq):  # noqa: F811
    """All of a commit's arrays in one tensor, the output between the inputs: nothing overlaps, nothing is refused."""
    lens, nodes, paths = [40, 21], [9, 5], [[0, 3, 7], [2]]
    bt = torch.tensor([[0, 1, 2], [3, 4, -1]], dtype=torch.int32)
    flat = torch.tensor([0, 9, 14] + lens + [-9, -9] + [3, 1] + [0, 3, 7, 2, 0, 0] + bt.flatten().tolist(), dtype=torch.int32).cuda()
    cu, sl, new, taken, path, tables = flat.split([3, 2, 2, 2, 6, 6])
    caches, want = (make_caches(5, 2, 64, ["fp8", "scale"]) for _ in range(2))
    before = flat.clone()
    kvq.kvq_tree_commit(caches, cu, tables.view(2, 3), sl, path.view(2, 3), taken, new)
    torch.cuda.synchronize()
    assert new.tolist() == [34, 17]
    before[5:7] = new
    assert torch.equal(flat, before)
    commit_plain(want, bt, [(n - m, p) for n, m, p in zip(lens, nodes, paths)])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(caches, want))


def test_commit_lengths_in_the_counts_are_refused(kvq):  # noqa: F811
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    taken = t([1])
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_tree_commit(make_caches(3, 2, 64, ["fp8"]), t([0, 4]), t([[0, 1]]), t([20]), t([[2]]), taken, taken)
    assert e.value.status == -7 and taken.tolist() == [1]


def test_fork_arrays_side_by_side(kvq):  # noqa: F811
    """The halves of one table, lengths and copies behind it: the outputs only touch the inputs."""
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, st = kvq.new_page_pool(12), t([0])
    flat = torch.full((2 * 3 + 3 * 3 + 2 + 3 + 3 + 6,), -1, dtype=torch.int32, device="cuda")
    tables, out, lens, out_lens, parents, copies = flat.split([6, 9, 2, 3, 3, 6])
    tables, out, copies = tables.view(2, 3), out.view(3, 3), copies.view(3, 2)
    lens.copy_(t([40, 20]))
    parents.copy_(t([1, 0, 0]))
    kvq.kvq_pages_alloc(pool, tables, t([0, 0]), lens, st)
    kvq.kvq_pages_fork(pool, tables, lens, parents, out, out_lens, copies, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and tables.tolist() == [[0, 1, 2], [3, 4, -1]]
    assert out.tolist() == [[3, 5, -1], [0, 1, 6], [0, 1, 7]] and out_lens.tolist() == [20, 40, 40]
    assert copies.tolist() == [[4, 5], [2, 6], [2, 7]]


@pytest.mark.parametrize("blocks,sources,beams,pages", [(300000, 512, 4096, 300), (40000, 16, 256, 2048), (20000, 4096, 4096, 3)])
def test_forks_at_full_width(kvq, blocks, sources, beams, pages):  # noqa: F811
    """As many rows as a call takes, and long tables, against the pool's rules in Python."""
    rng = random.Random(blocks)
    plain, mb = lib.Pool(blocks), pages + 2
    lens = [rng.choice((0, 16, rng.randint(1, 16 * pages), 16 * pages)) for _ in range(sources)]
    rows = [[-1] * mb for _ in range(sources)]
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, tables, st = kvq.new_page_pool(blocks), t(rows), t([0])
    assert plain.alloc(rows, [0] * sources, lens)
    kvq.kvq_pages_alloc(pool, tables, t([0] * sources), t(lens), st)
    parents = [rng.choice((-1, rng.randrange(sources), rng.randrange(sources), 0)) for _ in range(beams)]
    out, out_lens, copies = (torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((beams, mb), (beams,), (beams, 2)))
    kvq.kvq_pages_fork(pool, tables, t(lens), t(parents), out, out_lens, copies, st)
    want = plain.fork(rows, lens, parents, mb)
    torch.cuda.synchronize()
    assert int(st) == 0 and tables.tolist() == rows
    assert torch.equal(out.cpu(), torch.tensor(want[0], dtype=torch.int32))
    assert out_lens.tolist() == want[1] and copies.tolist() == want[2] and pool.tolist() == plain.words()
    # both sides given back: every page is free
    kvq.kvq_pages_free(pool, out, out_lens, torch.zeros_like(out_lens), st)
    kvq.kvq_pages_free(pool, tables, t(lens), t([0] * sources), st)
    torch.cuda.synchronize()
    assert int(st) == 0 and pool.tolist() == lib.Pool(blocks).words()


def test_largest_pool(kvq):  # noqa: F811
    """2^24 pages to 4096 rows of 4096, all of them; one more is refused; every second row given back and taken again."""
    n, B, mb = 1 << 24, 4096, 4097
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, st = torch.empty_like(kvq.new_page_pool(n)), t([0])
    kvq.kvq_pages_init(pool)
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    zero, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), 4096 * 16, dtype=torch.int32, device="cuda")
    kvq.kvq_pages_alloc(pool, tables, zero, lens, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and int(pool[1]) == 0 and bool((pool[4:4 + n] == 1).all()) and not bool(pool[4 + n:].any())
    want = torch.arange(n, dtype=torch.int32, device="cuda").view(B, 4096)
    assert torch.equal(tables[:, :4096], want) and bool((tables[:, 4096] == -1).all())
    more = lens.clone()
    more[7] += 1
    kvq.kvq_pages_alloc(pool, tables, lens, more, st)
    torch.cuda.synchronize()
    assert int(st) == kvq.KVQ_DEV_NO_PAGES and bool((tables[:, 4096] == -1).all())
    st.zero_()
    some = lens.clone()
    some[::2] = 0
    kvq.kvq_pages_free(pool, tables, lens, some, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and int(pool[1]) == n // 2 and bool((tables[::2, :4096] == -1).all())
    kvq.kvq_pages_alloc(pool, tables, some, lens, st)  # the lowest pages are those rows' again
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(tables[:, :4096], want)


def test_many_copies(kvq):  # noqa: F811
    n = 70000
    perm = torch.randperm(2 * n, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    cache = torch.arange(2 * n, dtype=torch.int32, device="cuda").view(2 * n, 1, 1, 1).expand(2 * n, 1, 16, 16).contiguous().view(torch.uint8).view(2 * n, 1, 16, 64)
    want = cache.clone()
    s, d = perm[:n].long().cuda(), perm[n:].long().cuda()
    want[d] = cache[s]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_copy_pages([cache], torch.stack([perm[:n], perm[n:]], 1).contiguous().cuda(), st)
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(cache, want)


def test_commits_of_many_sequences_and_long_paths(kvq):  # noqa: F811
    """65535 sequences of a page each; one sequence whose path has 4096 places."""
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B, st = 65535, t([0])
    cache = torch.randint(0, 256, (B, 1, 16, 64), generator=torch.Generator().manual_seed(2), dtype=torch.uint8).cuda()
    want = cache.clone()
    want[:, 0, 5], want[:, 0, 6] = cache[:, 0, 6], cache[:, 0, 9]  # nodes 1 and 4 of five behind five tokens
    new = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    kvq.kvq_tree_commit([cache], torch.arange(0, 5 * B + 1, 5, dtype=torch.int32, device="cuda"), torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                        torch.full_like(new, 10), t([[1, 4]]).repeat(B, 1), torch.full_like(new, 2), new, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and bool((new == 7).all()) and torch.equal(cache, want)
    pages = 600
    cache = torch.randint(0, 256, (pages, 2, 16, 64), generator=torch.Generator().manual_seed(3), dtype=torch.uint8).cuda()
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(4)).to(torch.int32)
    path = torch.randperm(9000, generator=torch.Generator().manual_seed(5))[:4096].sort().values
    want, pos = cache.clone(), torch.arange(4096)
    src, dst = 300 + path, 300 + pos
    want[order[dst // 16].long(), :, dst % 16] = cache[order[src // 16].long(), :, src % 16]
    new = t([-1])
    kvq.kvq_tree_commit([cache], t([0, 9000]), order[None].contiguous().cuda(), t([9300]), path.to(torch.int32)[None].contiguous().cuda(), t([4096]), new, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and int(new) == 4396 and torch.equal(cache, want)


@pytest.mark.parametrize("hq,hkv", [(513, 300), (2048, 256), (1, 1), (40, 5)])
def test_rope_of_many_heads(kvq, hq, hkv):  # noqa: F811
    c = Case(kvq, 9, hq, hkv, 64, lib.E4M3, axes=2, seed=hq)
    c.call()
    c.check()


def test_rope_axes_out_of_range_and_rows_of_a_wider_output(kvq):  # noqa: F811
    """An axis that there is not counts as axis 0; q_out as rows of a wider tensor, whose other columns stay."""
    c = Case(kvq, 70, 6, 2, 128, lib.E5M2, axes=3, seed=3)
    c.axis = c.axis.clone()
    given = c.axis.clone()
    given[::5], given[1::7] = 3, 255
    c.axis[::5], c.axis[1::7] = 0, 0
    wide = torch.full((70, 6 * 128 + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 16:16 + 6 * 128].unflatten(1, (6, 128))
    c.call(axis=given, q_out=out)
    c.out = out
    c.check()
    assert bool((wide[:, :16] == 5).all() & (wide[:, 16 + 768:] == 5).all())


@pytest.mark.parametrize("hq,hkv,seqs,fmt", [(2048, 256, [(70, 3), (33, 17)], lib.E4M3), (256, 256, [(200, 9)], lib.BF16),
                                             (8, 1, [(1 + i % 50, 1) for i in range(4096)], lib.E4M3),
                                             (16, 2, [(256 + i, 256) for i in range(40)], lib.E5M2)])
def test_trees_of_many_heads_and_sequences(kvq, hq, hkv, seqs, fmt):  # noqa: F811
    g = lib.OnGpu(kvq, lib.TreeBatch(seqs, hq, hkv, 64, fmt, seed=hq))
    g.call()
    g.check()
