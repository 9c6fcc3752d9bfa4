"""Bounded waits of the attention over trees that run out.

As in test_gpu_wait_timeout.py: a library built with the test hooks, whose CTA 0
never issues one copy, and with the waits cut to 2^16 polls.  The call reports
KVQ_DEV_WAIT_TIMEOUT and returns promptly, and the next one is right.  No GPU
fault is involved."""
import ctypes
import time

import pytest
import torch

import step_testlib as lib
from step_testlib import BF16, E4M3, PER_HEAD, PER_TOKEN_HEAD
from test_gpu_tree import kvq  # noqa: F401
from test_gpu_wait_timeout import tlib  # noqa: F401
from test_step_cpu import SIGNATURES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooked(tlib):  # noqa: F811
    for name, (res, args) in SIGNATURES.items():
        getattr(tlib, name).restype, getattr(tlib, name).argtypes = res, args
    return tlib


def call(lib_, g):
    """The call through the C ABI; how long it took."""
    b = g.b
    p = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None  # noqa: E731
    g.st.zero_()
    torch.cuda.synchronize()
    t0 = time.time()
    r = lib_.kvq_tree_attn(p(b.q), p(b.cu_d), b.q.shape[0], p(b.par), p(b.kc), p(b.vc), p(b.bt), b.bt.shape[1], p(b.sl), len(b.lens),
                           b.hq, b.hkv, b.dh, b.nb, 16, None, 0, p(b.ks), 0 if b.ks is None else b.ks.numel(), p(b.vs),
                           0 if b.vs is None else b.vs.numel(), b.gran, b.fmt, b.window, 0, p(g.ws), g.ws.numel(), p(g.out), p(g.st),
                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert r == 0
    torch.cuda.synchronize()
    return time.time() - t0


@pytest.mark.parametrize("seqs,hq,hkv,dh,fmt,gran", [
    ([(32768, 16)], 32, 8, 128, E4M3, PER_HEAD),              # a segment over many CTAs
    ([(300, 9)] * 200, 8, 2, 64, E4M3, PER_TOKEN_HEAD),       # several pieces a CTA
    ([(20000, 70)], 16, 8, 128, BF16, PER_HEAD)])             # rings of four blocks
@pytest.mark.parametrize("at", [0, 1, 2, 5, 12, 13])          # twice CTA 0's block, K or V
def test_copy_withheld(kvq, hooked, seqs, hq, hkv, dh, fmt, gran, at):  # noqa: F811
    g = lib.OnGpu(kvq, lib.TreeBatch(seqs, hq, hkv, dh, fmt, gran, seed=at))
    hooked.kvq_test_withhold_page(at)
    secs = call(hooked, g)
    hooked.kvq_test_withhold_page(-1)
    assert int(g.st.item()) == kvq.KVQ_DEV_WAIT_TIMEOUT
    assert secs < 30.0  # bounded: the waits gave up
    for what in ("after the timeout", "the call after"):
        g.out.fill_(3.0)
        call(hooked, g)
        g.check(what=what)
