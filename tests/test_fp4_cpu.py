"""What the 4-bit cache refuses, without a GPU: the C ABI on fake addresses
(every case returns before any CUDA call) and the binding's own checks."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # a 256-byte aligned fake address, never dereferenced


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_paged_gb300 as m
    return m


_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "kvq_fp4_write": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp]),
    "kvq_fp4_read": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _i32, _i64, _vp, _i32, _vp, _i32, _i32, _vp,
                            _vp, _i64, _vp, _vp]),
    "kvq_fp4_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "kvq_fp4_decode_attn": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i64, _i32, _vp, _i32, _vp, _i32, _i32,
                                   _i32, _i32, _vp, _sz, _vp, _vp, _vp]),
    "kvq_fp4_prefill_attn": (_i32, [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i64, _i32, _vp, _i32,
                                    _vp, _i32, _i32, _i32, _i32, _vp, _sz, _vp, _vp, _vp]),
}


@pytest.fixture(scope="module")
def clib(kvq):
    """The C ABI, past the binding."""
    raw = ctypes.CDLL(kvq.LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        getattr(raw, name).restype, getattr(raw, name).argtypes = res, args
    return raw


def test_exports(kvq, clib):
    from fp8_quantized_paged_gb300 import fp4
    text = open(os.path.join(ROOT, "include", "kvq_fp4.h")).read()
    declared = set(re.findall(r"KVQ_API\s+[\w\s\*]+?\b(kvq_\w+)\s*\(", text))
    assert declared == set(SIGNATURES)
    for name in declared:
        assert getattr(clib, name) is not None and getattr(kvq, name) is getattr(fp4, name)


def _call(clib, name, order, base, **kw):
    args = dict(base, **kw)
    assert set(args) == set(order)
    p = lambda x: ctypes.c_void_p(x) if x else None  # noqa: E731
    ptr = {"k", "v", "slots", "kc", "vc", "ks", "vs", "status", "bt", "starts", "cu", "ko", "vo", "q", "sl", "ws", "out", "stream"}
    return getattr(clib, name)(*[p(args[n]) if n in ptr else args[n] for n in order])


@pytest.fixture(scope="module")
def calls(clib):
    worder = "k v stride slots n hkv dh kc vc nb bs ks ksl vs vsl gran status stream".split()
    wbase = dict(k=A, v=A, stride=1024, slots=A, n=4, hkv=8, dh=128, kc=A, vc=A, nb=10, bs=16, ks=A, ksl=8, vs=A, vsl=8, gran=1,
                 status=0, stream=0)
    rorder = "kc vc nb bs hkv dh bt mb starts cu B n ks ksl vs vsl gran ko vo stride status stream".split()
    rbase = dict(kc=A, vc=A, nb=10, bs=16, hkv=8, dh=128, bt=A, mb=4, starts=0, cu=A, B=2, n=9, ks=A, ksl=8, vs=A, vsl=8, gran=1,
                 ko=A, vo=A, stride=1024, status=0, stream=0)
    tail = "sl B hq hkv dh nb bs ks ksl vs vsl gran window sinks ws wsb out status stream".split()
    tbase = dict(sl=A, B=2, hq=32, hkv=8, dh=128, nb=10, bs=16, ks=A, ksl=8, vs=A, vsl=8, gran=1, window=0, sinks=0, ws=A,
                 wsb=1 << 40, out=A, status=0, stream=0, kc=A, vc=A, bt=A, mb=4, q=A)
    return {"write": lambda **k: _call(clib, "kvq_fp4_write", worder, wbase, **k),
            "read": lambda **k: _call(clib, "kvq_fp4_read", rorder, rbase, **k),
            "decode": lambda **k: _call(clib, "kvq_fp4_decode_attn", "q kc vc bt mb".split() + tail, tbase, **k),
            "prefill": lambda **k: _call(clib, "kvq_fp4_prefill_attn", "q cu n maxq kc vc bt mb".split() + tail,
                                         dict(tbase, cu=A, n=20, maxq=10), **k)}


NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, ARG = -1, -2, -3, -4, -5, -7
COMMON = [(dict(kc=0), NULL), (dict(vc=0), NULL), (dict(ks=0), NULL), (dict(vs=0), NULL), (dict(dh=96), UNSUPPORTED),
          (dict(dh=256), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(gran=2), ARG), (dict(gran=-1), ARG), (dict(ksl=1), SHAPE),
          (dict(vsl=9), SHAPE), (dict(gran=0), SHAPE), (dict(nb=0), ARG), (dict(nb=-1), ARG), (dict(hkv=0), ARG),
          (dict(kc=A + 8), ALIGN), (dict(vc=A + 1), ALIGN), (dict(ks=A + 2), ALIGN), (dict(vs=A + 1), ALIGN),
          (dict(nb=1 << 62), SHAPE)]
ATTN = COMMON + [(dict(q=0), NULL), (dict(bt=0), NULL), (dict(sl=0), NULL), (dict(ws=0), NULL), (dict(out=0), NULL),
                 (dict(hq=30), SHAPE), (dict(hq=128), UNSUPPORTED), (dict(hq=0), ARG), (dict(B=0), ARG), (dict(mb=0), ARG),
                 (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(q=A + 8), ALIGN), (dict(out=A + 2), ALIGN),
                 (dict(ws=A + 128), ALIGN), (dict(bt=A + 2), ALIGN), (dict(sl=A + 1), ALIGN),
                 (dict(hq=257 * 2, hkv=257, ksl=257, vsl=257), UNSUPPORTED)]
CASES = {
    "write": COMMON + [(dict(k=0), NULL), (dict(v=0), NULL), (dict(slots=0), NULL), (dict(n=-1), ARG), (dict(stride=1023), SHAPE),
                       (dict(stride=1028), ALIGN), (dict(k=A + 8), ALIGN), (dict(slots=A + 4), ALIGN), (dict(stride=1 << 60), SHAPE),
                       (dict(hkv=70000, ksl=70000, vsl=70000, stride=1 << 30), UNSUPPORTED)],
    "read": COMMON + [(dict(bt=0), NULL), (dict(cu=0), NULL), (dict(ko=0), NULL), (dict(vo=0), NULL), (dict(n=-1), ARG),
                      (dict(B=0), ARG), (dict(mb=0), ARG), (dict(stride=1016), SHAPE), (dict(stride=1026), ALIGN),
                      (dict(ko=A + 4), ALIGN), (dict(cu=A + 1), ALIGN), (dict(starts=A + 3), ALIGN), (dict(stride=1 << 60), SHAPE)],
    "decode": ATTN + [(dict(B=5000), UNSUPPORTED), (dict(B=4096, mb=1 << 20), UNSUPPORTED),
                      (dict(B=4000, hkv=32, ksl=32, vsl=32), UNSUPPORTED),
                      (dict(B=1, hkv=1, hq=8, ksl=1, vsl=1, mb=1 << 27), UNSUPPORTED)],
    "prefill": ATTN + [(dict(cu=0), NULL), (dict(cu=A + 2), ALIGN), (dict(n=-1), ARG), (dict(maxq=-1), ARG),
                       (dict(B=70000), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED), (dict(n=1 << 40), UNSUPPORTED),
                       (dict(n=(1 << 30) + 1), UNSUPPORTED), (dict(B=65535, n=1 << 30, maxq=1 << 30), UNSUPPORTED)],
}


@pytest.mark.parametrize("name,over,want", [(n, o, w) for n, cs in CASES.items() for o, w in cs])
def test_abi_refusals(calls, name, over, want):
    assert calls[name](**over) == want


def test_abi_nothing_to_do(calls):
    assert calls["write"](n=0, k=0, v=0, slots=0) == 0
    assert calls["read"](n=0, ko=0, vo=0) == 0


def test_abi_prefill_of_no_queries(calls):
    assert calls["prefill"](n=0, q=0, out=0) == 0
    assert calls["prefill"](n=0, q=0, out=0, maxq=0) == 0
    assert calls["prefill"](n=0, q=0, out=0, cu=0) == NULL
    assert calls["prefill"](n=1, q=0) == NULL and calls["prefill"](n=1, out=0) == NULL


def test_workspace_size(kvq):
    f = kvq.kvq_fp4_workspace_size
    assert f(1, 8, 2, 64, 152) >= kvq.KVQ_WS_COUNTER_BYTES
    for bad in ((0, 8, 2, 64), (1, 0, 2, 64), (1, 8, 0, 64), (1, 9, 2, 64), (1, 8, 2, 96)):
        assert f(*bad, 152) == 0


# ------------------------------------------------------------------ the binding

B, HQ, HKV, DH, NB = 2, 8, 2, 64, 6


@pytest.fixture(scope="module")
def fp4(kvq):
    """The binding.  It looks at the device last, so a host tensor is refused for
    anything else that is wrong with it first, and no call reaches the library."""
    from fp8_quantized_paged_gb300 import fp4 as m
    return m


def _args(**over):
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d)  # noqa: E731
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    a = dict(q=z(B, HQ, DH), cu=z(B + 1, d=i32), maxq=1, kc=z(NB, HKV, 9 * DH, d=u8), vc=z(NB, HKV, 9 * DH, d=u8),
             bt=z(B, 3, d=i32), sl=z(B, d=i32), ks=z(HKV, d=f32), vs=z(HKV, d=f32), gran=1, window=0, sinks=0,
             ws=z(1 << 12, d=u8), out=z(B, HQ, DH), k=z(5, HKV, DH), v=z(5, HKV, DH), slots=z(5, d=torch.int64),
             starts=z(B, d=i32), ko=z(5, HKV, DH), vo=z(5, HKV, DH), st=None)
    return dict(a, **over)


def _run(m, op, a):
    if op == "write":
        m.kvq_fp4_write(a["k"], a["v"], a["slots"], a["kc"], a["vc"], a["ks"], a["vs"], a["gran"], dev_status=a["st"])
    elif op == "read":
        m.kvq_fp4_read(a["kc"], a["vc"], a["bt"], a["starts"], a["cu"], a["ks"], a["vs"], a["gran"], a["ko"], a["vo"], dev_status=a["st"])
    elif op == "decode":
        m.kvq_fp4_decode_attn(a["q"], a["kc"], a["vc"], a["bt"], a["sl"], a["ks"], a["vs"], a["gran"], a["window"], a["sinks"],
                              a["ws"], a["out"], dev_status=a["st"])
    else:
        m.kvq_fp4_prefill_attn(a["q"], a["cu"], a["maxq"], a["kc"], a["vc"], a["bt"], a["sl"], a["ks"], a["vs"], a["gran"],
                               a["window"], a["sinks"], a["ws"], a["out"], dev_status=a["st"])


def t(*s, d=torch.bfloat16):
    return torch.zeros(s, dtype=d)


BOTH = [(dict(kc=t(NB, HKV, 9 * DH)), ARG, "k_cache"), (dict(kc=t(NB, 9 * DH, d=torch.uint8)), SHAPE, "caches"), (dict(vc=t(NB + 1, HKV, 9 * DH, d=torch.uint8)), SHAPE, "v_cache"),
        (dict(kc=t(NB, HKV, 16, DH, d=torch.uint8)), SHAPE, "caches"), (dict(kc=t(NB, HKV, 500, d=torch.uint8)), SHAPE, "page"),
        (dict(kc=t(NB, 9 * DH, HKV, d=torch.uint8).transpose(1, 2)), SHAPE, "contiguous"),
        (dict(ks=t(HKV)), ARG, "k_scale"), (dict(vs=t(HKV, d=torch.float64)), ARG, "v_scale"),
        (dict(st=t(1, d=torch.int64)), ARG, "dev_status"), (dict(st=t(0, d=torch.int32)), ARG, "dev_status")]
MORE = {
    "write": [(dict(k=t(5, HKV, DH, d=torch.float16)), ARG, "k must"), (dict(v=t(5, HKV, DH + 1)), SHAPE, "v must"),
              (dict(v=t(4, HKV, DH)), SHAPE, "v must"), (dict(k=t(5, DH, HKV).transpose(1, 2)), SHAPE, "dense"),
              (dict(k=t(5, 2, HKV, DH)[:, 0]), SHAPE, "row distance"), (dict(slots=t(5, d=torch.int32)), ARG, "slot_mapping"),
              (dict(slots=t(4, d=torch.int64)), SHAPE, "slot_mapping"), (dict(kc=t(NB, HKV + 1, 9 * DH, d=torch.uint8),
                                                                              vc=t(NB, HKV + 1, 9 * DH, d=torch.uint8)), SHAPE, "KV heads"),
              (dict(k=t(5, HKV, 128), v=t(5, HKV, 128)), SHAPE, "page")],
    "read": [(dict(ko=t(5, HKV, DH, d=torch.float32)), ARG, "k_out"), (dict(vo=t(6, HKV, DH)), SHAPE, "v_out"),
             (dict(ko=t(5, 2, HKV, DH)[:, 1]), SHAPE, "row distance"), (dict(cu=t(B, d=torch.int32)), SHAPE, "cu_lens"),
             (dict(starts=t(B + 1, d=torch.int32)), SHAPE, "starts"), (dict(bt=t(B, 3, d=torch.int64)), ARG, "block_tables")],
    "decode": [(dict(q=t(B, HQ, 128)), SHAPE, "page"), (dict(q=t(B, HQ, DH, d=torch.float16)), ARG, "q must"),
               (dict(out=t(B, HQ, DH + 2)), SHAPE, "out"), (dict(out=t(B, HQ, DH, d=torch.float32)), ARG, "out"),
               (dict(bt=t(B + 1, 3, d=torch.int32)), SHAPE, "block_tables"), (dict(bt=t(B, 3)), ARG, "block_tables"),
               (dict(sl=t(B + 1, d=torch.int32)), SHAPE, "seq_lens"), (dict(ws=t(99, d=torch.float32)), ARG, "workspace"),
               (dict(q=t(HQ, B, DH).transpose(0, 1)), SHAPE, "contiguous")],
}
MORE["prefill"] = MORE["decode"][:5] + [(dict(cu=t(B, d=torch.int32)), SHAPE, "cu_q_lens"), (dict(cu=t(B + 1, d=torch.int64)), ARG, "cu_q_lens"),
                                        (dict(ws=t(99, d=torch.float32)), ARG, "workspace")]


@pytest.mark.parametrize("op,over,status,word", [(op, *c) for op in MORE for c in BOTH + MORE[op]])
def test_binding_refusals(fp4, op, over, status, word):
    with pytest.raises(fp4.KvqError) as e:
        _run(fp4, op, _args(**over))
    assert e.value.status == status and word in str(e.value)


def test_binding_wants_cuda_tensors(kvq, fp4):
    for op in ("write", "read", "decode", "prefill"):
        with pytest.raises(kvq.KvqError) as e:
            _run(fp4, op, _args())
        assert e.value.status == ARG and "CUDA" in str(e.value)


def test_binding_arguments(fp4):
    a = _args()
    pos = (a["k"], a["v"], a["slots"], a["kc"], a["vc"], a["ks"], a["vs"])
    for call in (lambda: fp4.kvq_fp4_write(*pos), lambda: fp4.kvq_fp4_write(*pos, 1, None, None, 3),
                 lambda: fp4.kvq_fp4_write(*pos, 1, other=3), lambda: fp4.kvq_fp4_write(*pos, 1, k=a["k"]),
                 lambda: fp4.kvq_fp4_write(7, *pos[1:], 1), lambda: fp4.kvq_fp4_write(None, *pos[1:], 1)):
        with pytest.raises(TypeError):
            call()
    for bad in ("one", 1.5, None, 1 << 40, -(1 << 70)):
        with pytest.raises(fp4.KvqError) as e:
            fp4.kvq_fp4_write(*pos, bad)
        assert e.value.status == ARG and "scale_granularity" in str(e.value)
    # by name, in any order: as far as the device check
    with pytest.raises(fp4.KvqError) as e:
        fp4.kvq_fp4_write(scale_granularity=1, v_scale=a["vs"], k=a["k"], v=a["v"], slot_mapping=a["slots"], k_cache=a["kc"],
                          v_cache=a["vc"], k_scale=a["ks"], stream=None, dev_status=None)
    assert "CUDA" in str(e.value)
