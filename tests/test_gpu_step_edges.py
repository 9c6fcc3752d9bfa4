"""Ordinary calls of the step's operators at the edges of what they take."""
import pytest
import torch

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
