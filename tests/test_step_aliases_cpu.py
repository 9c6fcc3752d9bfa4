"""Outputs that lie in inputs are refused, without a GPU (fake addresses, never dereferenced)."""
import pytest

from test_step_cpu import A, ARG, call, clib, kvq  # noqa: F401

# an ordinary call's arrays, apart from each other: 2 sequences, tables of 4 pages, paths of 7
APART = dict(cu=A, bt=A + 256, sl=A + 512, path=A + 768, taken=A + 1024)
LAST = dict(cu=A + 8, bt=A + 256 + 28, sl=A + 512 + 4, path=A + 768 + 52, taken=A + 1024 + 4)  # their last words


@pytest.mark.parametrize("name", sorted(APART))
def test_commit_lengths_in_an_input(clib, name):  # noqa: F811
    """new_lens is written while the other caches' warps still read: an input as the output would move some layers only."""
    for new in (APART[name], LAST[name], APART[name] - 4):
        assert call(clib, "kvq_tree_commit", **APART, new=new) == ARG



# a fork of 2 sequences into 3, tables of 4 pages, a pool of 10
FORK = dict(pool=A, bt=A + 256, sl=A + 512, parents=A + 768, out=A + 1024, ol=A + 1280, copies=A + 1536)
BYTES = dict(pool=4 * 15, bt=4 * 8, sl=4 * 2, parents=4 * 3, out=4 * 12, ol=4 * 3, copies=4 * 6)


@pytest.mark.parametrize("out,other", [(o, i) for o in ("out", "ol", "copies") for i in FORK if i != o])
def test_fork_outputs_apart(clib, out, other):  # noqa: F811
    """An output in an input, in the pool or in another output, whole or by one word."""
    for at in (FORK[other], FORK[other] + BYTES[other] - 4, FORK[other] - BYTES[out] + 4):
        assert call(clib, "kvq_pages_fork", **dict(FORK, **{out: at})) == ARG
