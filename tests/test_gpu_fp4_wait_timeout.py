"""Bounded waits of the 4-bit cache's attentions that run out.

As in test_gpu_wait_timeout.py: a library built with the test hooks, whose CTA 0
never issues one copy, and with the waits cut to 2^16 polls.  The call reports
KVQ_DEV_WAIT_TIMEOUT and returns promptly, and once the counters are cleared the
next one is right.  No GPU fault is involved."""
import ctypes
import time

import numpy as np
import pytest
import torch

import fp4_testlib as f4
from test_fp4_cpu import SIGNATURES
from test_gpu_fp4 import OnGpu, kvq  # noqa: F401
from test_gpu_wait_timeout import tlib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooked(tlib):  # noqa: F811
    for name, (res, args) in SIGNATURES.items():
        getattr(tlib, name).restype, getattr(tlib, name).argtypes = res, args
    return tlib


def call(lib, g, op, window, sinks):
    """The call through the C ABI; how long it took."""
    b = g.b
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    pages = [p(g.kc), p(g.vc), p(g.bt), g.bt.shape[1], p(g.sl), len(b.lens), b.hq, b.hkv, b.dh, b.nb, 16, p(g.ks), g.ks.numel(),
             p(g.vs), g.vs.numel(), b.gran, window, sinks, p(g.ws), g.ws.numel(), p(g.out), p(g.st),
             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)]
    g.st.zero_()
    torch.cuda.synchronize()
    t0 = time.time()
    if op == "decode":
        r = lib.kvq_fp4_decode_attn(p(g.dq), *pages)
    else:
        r = lib.kvq_fp4_prefill_attn(p(g.dq), p(g.dcu), g.q.shape[0], int(np.diff(g.cu).max()), *pages)
    assert r == 0
    torch.cuda.synchronize()
    return time.time() - t0


def times_out_then_recovers(kvq, lib, g, op, at, window=0, sinks=0, also=0):  # noqa: F811
    lib.kvq_test_withhold_page(at)
    secs = call(lib, g, op, window, sinks)
    lib.kvq_test_withhold_page(-1)
    assert int(g.st.item()) == kvq.KVQ_DEV_WAIT_TIMEOUT | also
    assert secs < 30.0  # bounded: the waits gave up
    g.ws[:kvq.KVQ_WS_COUNTER_BYTES].zero_()
    for what in ("after the timeout", "the call after"):  # a completed call leaves the counters zero
        g.out.fill_(3.0)
        call(lib, g, op, window, sinks)
        g.check(window, sinks, what, status=also)
    return secs


@pytest.mark.parametrize("lens,hq,hkv,dh", [
    ([1600, 1000], 32, 8, 128),        # a CTA a segment
    ([32768], 8, 8, 64),               # a segment over many CTAs
    ([4096] * 4, 32, 8, 128),          # units of two heads
    ([2300] * 20, 8, 8, 128)])         # of eight
@pytest.mark.parametrize("at", [0, 3, 10])
def test_decode_copy_withheld(kvq, hooked, lens, hq, hkv, dh, at):  # noqa: F811
    g = OnGpu(kvq, f4.Batch(len(lens) + at, lens, hq, hkv, dh), [1] * len(lens))
    times_out_then_recovers(kvq, hooked, g, "decode", at)


@pytest.mark.parametrize("lens,counts,hq,hkv,dh", [
    ([700], [700], 4, 1, 128),                 # two tiles a CTA
    ([700, 90], [90, 9], 8, 2, 64),            # ragged
    ([20000], [4], 32, 8, 128)])               # keys shared out
@pytest.mark.parametrize("at", [0, 1, 2, 5])
def test_prefill_copy_withheld(kvq, hooked, lens, counts, hq, hkv, dh, at):  # noqa: F811
    b = f4.Batch(sum(lens) + at, lens, hq, hkv, dh)
    g = OnGpu(kvq, b, counts)
    times_out_then_recovers(kvq, hooked, g, "prefill", at)


def test_decode_drain_after_bad_pages(kvq, hooked):  # noqa: F811
    """Slots that held a good page and then a bad one are done with: the exit waits for
    none of them (each such wait used up all its polls, some 40 times the one withheld copy's)."""
    b = f4.Batch(9, [32768], 8, 8, 64)  # CTA 0: units 0 .. 106, rings of 56 slots in all
    assert b.table.shape[1] == 2048
    b.table[0, 40:2048:2] = -1
    b.table[0, 41:107] = -1
    g = OnGpu(kvq, b, [1])
    bad = times_out_then_recovers(kvq, hooked, g, "decode", 106, also=kvq.KVQ_DEV_BAD_BLOCK)
    b = f4.Batch(9, [32768], 8, 8, 64)
    good = times_out_then_recovers(kvq, hooked, OnGpu(kvq, b, [1]), "decode", 106)
    assert bad < 8 * good + 0.5, (bad, good)
