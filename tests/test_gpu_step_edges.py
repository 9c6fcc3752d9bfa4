"""Ordinary calls of the step's operators at the edges of what they take."""
import random

import pytest
import torch

import step_testlib as lib
from test_gpu_pages import commit_plain, kvq, make_caches  # noqa: F401

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
