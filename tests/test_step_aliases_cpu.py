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

