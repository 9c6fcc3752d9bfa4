"""What the operators around a serving step refuse, without a GPU: the C ABI on fake
addresses (every case returns before any CUDA call) and the binding's own checks."""
import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # a 256-byte aligned fake address, never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, ARG = -1, -2, -3, -4, -5, -7
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_f32, _u32 = ctypes.c_float, ctypes.c_uint


class Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("row_bytes", ctypes.c_int32), ("sub_bytes", ctypes.c_int32)]


# name: (result, [(argument, type, what an ordinary call gives)])
CALLS = {
    "kvq_rope_write": (_i32, [
        ("q", _vp, A), ("q_stride", _i64, 4096), ("k", _vp, A), ("k_stride", _i64, 1024), ("v", _vp, A), ("v_stride", _i64, 1024),
        ("n", _i64, 5), ("hq", _i32, 32), ("hkv", _i32, 8), ("dh", _i32, 128), ("pos", _vp, A), ("axes", _i32, 1), ("turns", _vp, A),
        ("axis", _vp, 0), ("pairs", _i32, 64), ("inter", _i32, 0), ("wq", _vp, A), ("wk", _vp, A), ("eps", _f32, 1e-6),
        ("slots", _vp, A), ("kc", _vp, A), ("vc", _vp, A), ("nb", _i64, 10), ("bs", _i32, 16), ("ks", _vp, A), ("ksl", _i32, 8),
        ("vs", _vp, A), ("vsl", _i32, 8), ("gran", _i32, 1), ("fmt", _i32, 1), ("out", _vp, A + 4096), ("ostride", _i64, 4096),
        ("status", _vp, 0), ("stream", _vp, 0)]),
    "kvq_tree_workspace_size": (_sz, [("hq", _i32, 32), ("hkv", _i32, 8), ("dh", _i32, 128), ("sms", _i32, 152)]),
    "kvq_tree_attn": (_i32, [
        ("q", _vp, A), ("cu", _vp, A), ("n", _i64, 20), ("parents", _vp, A), ("kc", _vp, A), ("vc", _vp, A), ("bt", _vp, A),
        ("mb", _i32, 4), ("sl", _vp, A), ("B", _i32, 2), ("hq", _i32, 32), ("hkv", _i32, 8), ("dh", _i32, 128), ("nb", _i64, 10),
        ("bs", _i32, 16), ("qs", _vp, 0), ("qsl", _i32, 0), ("ks", _vp, A), ("ksl", _i32, 8), ("vs", _vp, A), ("vsl", _i32, 8),
        ("gran", _i32, 1), ("fmt", _i32, 1), ("window", _i32, 0), ("flags", _u32, 0), ("ws", _vp, A), ("wsb", _sz, 1 << 40),
        ("out", _vp, A), ("status", _vp, 0), ("stream", _vp, 0)]),
    "kvq_tree_commit": (_i32, [
        ("caches", ctypes.POINTER(Rows), None), ("nc", _i32, 2), ("nb", _i64, 10), ("hkv", _i32, 8), ("bs", _i32, 16), ("cu", _vp, A),
        ("bt", _vp, A), ("mb", _i32, 4), ("sl", _vp, A), ("B", _i32, 2), ("path", _vp, A), ("most", _i32, 7), ("taken", _vp, A),
        ("new", _vp, A + 64), ("status", _vp, 0), ("stream", _vp, 0)]),
    "kvq_copy_pages": (_i32, [
        ("caches", ctypes.POINTER(Rows), None), ("nc", _i32, 2), ("nb", _i64, 10), ("hkv", _i32, 8), ("bs", _i32, 16),
        ("copies", _vp, A), ("n", _i32, 3), ("status", _vp, 0), ("stream", _vp, 0)]),
    "kvq_pages_init": (_i32, [("pool", _vp, A), ("nb", _i64, 10), ("stream", _vp, 0)]),
    "kvq_pages_alloc": (_i32, [("pool", _vp, A), ("nb", _i64, 10), ("bt", _vp, A), ("mb", _i32, 4), ("old", _vp, A), ("new", _vp, A),
                               ("B", _i32, 2), ("status", _vp, 0), ("stream", _vp, 0)]),
    "kvq_pages_fork": (_i32, [("pool", _vp, A), ("nb", _i64, 10), ("bt", _vp, A), ("sl", _vp, A), ("ns", _i32, 2), ("mb", _i32, 4),
                              ("parents", _vp, A), ("no", _i32, 3), ("out", _vp, A + 256), ("ol", _vp, A + 512),
                              ("copies", _vp, A + 768), ("status", _vp, 0), ("stream", _vp, 0)]),
}
CALLS["kvq_pages_free"] = CALLS["kvq_pages_alloc"]
SIGNATURES = {n: (r, [t for _, t, _ in a]) for n, (r, a) in CALLS.items()}


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_paged_gb300 as m
    return m


@pytest.fixture(scope="module")
def clib(kvq):
    """The C ABI, past the binding."""
    raw = ctypes.CDLL(kvq.LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        getattr(raw, name).restype, getattr(raw, name).argtypes = res, args
    return raw


def test_exports(kvq, clib):
    from fp8_quantized_paged_gb300 import step
    text = open(os.path.join(ROOT, "include", "kvq_step.h")).read()
    declared = set(re.findall(r"KVQ_API\s+[\w\s\*]+?\b(kvq_\w+)\s*\(", text))
    assert declared == set(SIGNATURES)
    for name in declared:
        assert getattr(clib, name) is not None and getattr(kvq, name) is getattr(step, name)
    for name, want in (("KVQ_DEV_NO_PAGES", kvq.KVQ_DEV_NO_PAGES), ("KVQ_DEV_BAD_TREE", kvq.KVQ_DEV_BAD_TREE),
                       ("KVQ_TREE_MAX_NODES", kvq.KVQ_TREE_MAX_NODES), ("KVQ_POOL_HEADER", step.KVQ_POOL_HEADER)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == want


def call(clib, name, **over):
    args = {n: v for n, _, v in CALLS[name][1]}
    assert set(over) <= set(args)
    args.update(over)
    if args.get("caches", 0) is None:
        args["caches"] = (Rows * max(1, args["nc"]))(*(Rows(A + 4096 * i, 128, 0) for i in range(max(0, args["nc"]))))
    out = []
    for n, t, _ in CALLS[name][1]:
        out.append((_vp(args[n]) if args[n] else None) if t is _vp else args[n])
    return getattr(clib, name)(*out)


CACHE = [(dict(kc=0), NULL), (dict(vc=0), NULL), (dict(ks=0), NULL), (dict(vs=0), NULL), (dict(dh=96), UNSUPPORTED),
         (dict(dh=256), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(gran=3), ARG), (dict(gran=-1), ARG), (dict(fmt=3), ARG),
         (dict(fmt=-1), ARG), (dict(ksl=1), SHAPE), (dict(vsl=9), SHAPE), (dict(gran=0), SHAPE), (dict(gran=2), SHAPE),
         (dict(nb=0), ARG), (dict(nb=-1), ARG), (dict(hkv=0), ARG), (dict(kc=A + 8), ALIGN), (dict(vc=A + 1), ALIGN),
         (dict(ks=A + 2), ALIGN), (dict(vs=A + 1), ALIGN), (dict(gran=2, ksl=1280, vsl=1280, ks=A + 4), ALIGN)]
ROWS = [(dict(nc=-1), ARG), (dict(nb=0), ARG), (dict(hkv=0), ARG), (dict(hkv=70000), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
        (dict(nb=1 << 62), SHAPE)] + [
    (dict(nc=1, caches=(Rows * 1)(Rows(*r))), want) for r, want in (
        ((0, 128, 0), NULL), ((A, 0, 0), SHAPE), ((A, 126, 0), SHAPE), ((A, 516, 0), SHAPE), ((A, 64, -4), SHAPE), ((A, 64, 6), SHAPE),
        ((A, 64, 516), SHAPE), ((A + 8, 128, 0), ALIGN))]
POOL = [(dict(pool=0), NULL), (dict(nb=0), ARG), (dict(nb=(1 << 24) + 1), UNSUPPORTED), (dict(pool=A + 2), ALIGN)]
TABLES = POOL + [(dict(bt=0), NULL), (dict(old=0), NULL), (dict(new=0), NULL), (dict(mb=0), ARG), (dict(mb=1 << 28), UNSUPPORTED),
                 (dict(B=-1), ARG), (dict(B=4097), UNSUPPORTED), (dict(bt=A + 1), ALIGN), (dict(old=A + 2), ALIGN), (dict(new=A + 3), ALIGN)]
REFUSED = {
    "kvq_rope_write": CACHE + [
        (dict(n=-1), ARG), (dict(hq=0), ARG), (dict(axes=0), ARG), (dict(axes=17), UNSUPPORTED), (dict(pairs=-8), ARG),
        (dict(pairs=60), SHAPE), (dict(pairs=72), SHAPE), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(turns=0), NULL),
        (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(out=0), NULL), (dict(slots=0), NULL), (dict(pos=0), NULL),
        (dict(q_stride=4088), SHAPE), (dict(k_stride=1016), SHAPE), (dict(v_stride=0), SHAPE), (dict(ostride=4095), SHAPE),
        (dict(q_stride=4100), ALIGN), (dict(k_stride=1028), ALIGN), (dict(ostride=4097), ALIGN),
        (dict(out=A, ostride=8192), SHAPE),  # in place, but with another stride
        (dict(q=A + 8), ALIGN), (dict(k=A + 2), ALIGN), (dict(out=A + 4), ALIGN), (dict(wq=A + 8), ALIGN), (dict(wk=A + 2), ALIGN),
        (dict(slots=A + 4), ALIGN), (dict(turns=A + 4), ALIGN), (dict(pos=A + 2), ALIGN), (dict(fmt=0, gran=2), UNSUPPORTED),
        (dict(hq=65530, q_stride=1 << 24, ostride=1 << 24), UNSUPPORTED), (dict(nb=1 << 60), SHAPE)],
    "kvq_tree_attn": CACHE + [
        (dict(n=-1), ARG), (dict(B=0), ARG), (dict(hq=0), ARG), (dict(mb=0), ARG), (dict(window=-1), ARG), (dict(flags=2), ARG),
        (dict(flags=1), NULL), (dict(flags=1, fmt=0, qs=A, qsl=32), UNSUPPORTED), (dict(qs=A, qsl=1), SHAPE),
        (dict(qs=A + 2, qsl=32), ALIGN), (dict(q=0), NULL), (dict(cu=0), NULL), (dict(bt=0), NULL), (dict(sl=0), NULL),
        (dict(ws=0), NULL), (dict(out=0), NULL), (dict(hq=30), SHAPE), (dict(hq=72), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
        (dict(hkv=257, hq=257, ksl=257, vsl=257), UNSUPPORTED), (dict(mb=1 << 26), UNSUPPORTED), (dict(n=(1 << 30) + 1), UNSUPPORTED),
        (dict(n=4096, B=4096, mb=16 * 1024), UNSUPPORTED), (dict(nb=1 << 24), UNSUPPORTED), (dict(q=A + 8), ALIGN),
        (dict(out=A + 2), ALIGN), (dict(ws=A + 128), ALIGN), (dict(bt=A + 2), ALIGN), (dict(sl=A + 1), ALIGN), (dict(cu=A + 3), ALIGN),
        (dict(parents=A + 2), ALIGN)],
    "kvq_tree_commit": ROWS + [
        (dict(cu=0), NULL), (dict(bt=0), NULL), (dict(sl=0), NULL), (dict(path=0), NULL), (dict(taken=0), NULL), (dict(new=0), NULL),
        (dict(B=-1), ARG), (dict(most=-1), ARG), (dict(mb=0), ARG), (dict(B=65536), UNSUPPORTED), (dict(most=4097), UNSUPPORTED),
        (dict(mb=1 << 28), UNSUPPORTED), (dict(cu=A + 1), ALIGN), (dict(path=A + 2), ALIGN), (dict(new=A + 66), ALIGN),
        (dict(new=A), ARG),  # the lengths in place
        (dict(nc=3, caches=(Rows * 3)(Rows(A, 64, 8), Rows(A + 64, 64, 8), Rows(A, 64, 8))), ARG),  # a cache twice
        (dict(nc=2, caches=(Rows * 2)(Rows(A, 64, 8), Rows(A, 4, 0))), ARG), (dict(nc=1025), UNSUPPORTED)],
    "kvq_copy_pages": ROWS + [(dict(copies=0), NULL), (dict(n=-1), ARG), (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(copies=A + 2), ALIGN)],
    "kvq_pages_init": POOL,
    "kvq_pages_alloc": TABLES,
    "kvq_pages_free": TABLES,
    "kvq_pages_fork": POOL + [
        (dict(bt=0), NULL), (dict(sl=0), NULL), (dict(parents=0), NULL), (dict(out=0), NULL), (dict(ol=0), NULL), (dict(copies=0), NULL),
        (dict(mb=0), ARG), (dict(ns=-1), ARG), (dict(no=-1), ARG), (dict(ns=4097), UNSUPPORTED), (dict(no=4097), UNSUPPORTED),
        (dict(parents=A + 2), ALIGN), (dict(copies=A + 770), ALIGN), (dict(out=A), ARG), (dict(ol=A, sl=A, bt=A + 1024), ARG)],
}


@pytest.mark.parametrize("name,over,want", [(n, o, w) for n, cs in REFUSED.items() for o, w in cs])
def test_abi_refusals(clib, name, over, want):
    assert call(clib, name, **over) == want


def test_abi_nothing_to_do(clib):
    assert call(clib, "kvq_rope_write", n=0, q=0, k=0, v=0, out=0, slots=0, pos=0) == 0
    assert call(clib, "kvq_tree_attn", n=0, q=0, out=0) == 0
    assert call(clib, "kvq_tree_commit", B=0, cu=0, bt=0, sl=0, path=0, taken=0, new=0) == 0
    assert call(clib, "kvq_copy_pages", n=0, copies=0) == 0
    assert call(clib, "kvq_pages_alloc", B=0, bt=0, old=0, new=0) == 0
    assert call(clib, "kvq_pages_free", B=0, bt=0, old=0, new=0) == 0
    assert call(clib, "kvq_pages_fork", no=0, parents=0, out=0, ol=0, copies=0) == 0


def test_workspace_size(kvq):
    f = kvq.kvq_tree_workspace_size
    # two states a CTA of 128 rows: maximum and sum, and head_dim sums
    assert f(32, 8, 128, 152) >= 152 * 2 * 128 * (8 + 4 * 128) and f(8, 2, 64, 152) < f(32, 8, 128, 152) == f(8, 8, 128, 152)
    for bad in ((0, 8, 64), (8, 0, 64), (9, 2, 64), (18, 2, 64), (8, 2, 96)):
        assert f(*bad, 152) == 0


def test_rope_turns(kvq):
    """round(2^64 f / 2 pi) modulo 2^64, as signed words."""
    f = [1.0, 1e-4, 2 * math.pi * 0.75, 0.0, 500.0, -1.0]
    got = kvq.rope_turns(f, device="cpu")
    assert got.dtype == torch.int64
    for x, g in zip(f, got.tolist()):
        d = (g - round(x / (2 * math.pi) * 2.0 ** 64)) % (1 << 64)
        assert d == 0 and -(1 << 63) <= g < 1 << 63
    assert torch.equal(kvq.rope_turns(torch.tensor(f, dtype=torch.float64), device="cpu"), got)


def test_new_page_pool(kvq):
    for n in (1, 31, 32, 33, 1000):
        p = kvq.new_page_pool(n, device="cpu")
        assert p.numel() == 4 + n + (n + 31) // 32 and p[:4].tolist() == [0, n, 0, 0] and not p[4:4 + n].any()
        bits = [(w >> i) & 1 for w in (p[4 + n:].tolist()) for i in range(32)]
        assert bits == [1] * n + [0] * (len(bits) - n)
    for n in (0, -1, (1 << 24) + 1):
        with pytest.raises(kvq.KvqError):
            kvq.new_page_pool(n, device="cpu")


# ------------------------------------------------------------------ the binding

B, HQ, HKV, DH, NB, N = 2, 8, 2, 64, 6, 5


@pytest.fixture(scope="module")
def step(kvq):
    """The binding.  It looks at the device last, so a host tensor is refused for
    anything else that is wrong with it first, and no call reaches the library."""
    from fp8_quantized_paged_gb300 import step as m
    return m


def t(*s, d=torch.bfloat16):
    return torch.zeros(s, dtype=d)


i32, u8, f32, i64 = torch.int32, torch.uint8, torch.float32, torch.int64


def arguments(op):
    kc, vc = t(NB, HKV, 16, DH, d=u8), t(NB, HKV, 16, DH, d=u8)
    pool = t(4 + 40 + 2, d=i32)
    return {
        "kvq_rope_write": dict(q=t(N, HQ, DH), k=t(N, HKV, DH), v=t(N, HKV, DH), positions=t(N, d=i32), turns=t(32, d=i64), axis=None,
                               q_weight=t(DH), k_weight=None, eps=1e-6, interleaved=False, slot_mapping=t(N, d=i64), k_cache=kc, v_cache=vc,
                               k_scale=t(HKV, d=f32), v_scale=t(HKV, d=f32), scale_granularity=1, fmt=1, q_out=t(N, HQ, DH)),
        "kvq_tree_attn": dict(q=t(N, HQ, DH), cu_q_lens=t(B + 1, d=i32), parents=t(N, d=i32), k_cache=kc, v_cache=vc,
                              block_tables=t(B, 3, d=i32), seq_lens=t(B, d=i32), k_scale=t(HKV, d=f32), v_scale=t(HKV, d=f32),
                              scale_granularity=1, fmt=1, sliding_window=0, workspace=t(64, d=u8), out=t(N, HQ, DH)),
        "kvq_tree_commit": dict(caches=[kc, vc], cu_q_lens=t(B + 1, d=i32), block_tables=t(B, 3, d=i32), seq_lens=t(B, d=i32),
                                accepted=t(B, 4, d=i32), num_accepted=t(B, d=i32), new_lens=t(B, d=i32)),
        "kvq_copy_pages": dict(caches=[kc, vc], copies=t(3, 2, d=i32)),
        "kvq_pages_init": dict(pool=pool),
        "kvq_pages_alloc": dict(pool=pool, block_tables=t(B, 3, d=i32), old_lens=t(B, d=i32), new_lens=t(B, d=i32)),
        "kvq_pages_free": dict(pool=pool, block_tables=t(B, 3, d=i32), old_lens=t(B, d=i32), new_lens=t(B, d=i32)),
        "kvq_pages_fork": dict(pool=pool, block_tables=t(B, 3, d=i32), seq_lens=t(B, d=i32), parents=t(4, d=i32),
                               out_tables=t(4, 3, d=i32), out_lens=t(4, d=i32), copies=t(4, 2, d=i32)),
    }[op]


STATUS = [(dict(dev_status=t(1, d=i64)), ARG, "dev_status"), (dict(dev_status=t(0, d=i32)), ARG, "dev_status")]
PAGES = [(dict(k_cache=t(NB, HKV, 16, DH)), ARG, "k_cache"), (dict(v_cache=t(NB + 1, HKV, 16, DH, d=u8)), SHAPE, "v_cache"),
         (dict(k_cache=t(NB, HKV, 8, DH, d=u8)), SHAPE, "k_cache"), (dict(k_cache=t(NB, 16, HKV, DH, d=u8).transpose(1, 2)), SHAPE, "contiguous"),
         (dict(fmt=7), ARG, "format"), (dict(k_scale=t(HKV)), ARG, "k_scale"), (dict(v_scale=t(HKV, d=torch.float64)), ARG, "v_scale"),
         (dict(q=t(N, HQ, 128)), SHAPE, ""), (dict(q=t(N, HQ, DH, d=torch.float16)), ARG, "q must"), (dict(q=t(N, HQ * DH)), SHAPE, "q ")]
LIST = [(dict(caches=[]), ARG, "caches"), (dict(caches=[t(NB, HKV, 16, DH, d=u8), t(NB + 1, HKV, 16, DH, d=u8)]), SHAPE, "same blocks"),
        (dict(caches=[t(NB, HKV, 16, 96, d=u8)]), SHAPE, "a cache"), (dict(caches=[t(NB, HKV, 500, d=u8)]), SHAPE, "a cache"),
        (dict(caches=[t(NB, HKV, 16, DH, d=f32)]), SHAPE, "a cache"), (dict(caches=[t(NB, 16, HKV, DH, d=u8).transpose(1, 2)]), SHAPE, "")]
TAKEN = [(dict(pool=t(38, d=i32)), SHAPE, "pool"), (dict(pool=t(4, d=i32)), SHAPE, "pool"), (dict(pool=t(46, d=i64)), ARG, "pool")]
LENS = [(dict(block_tables=t(B, 3, d=i64)), ARG, "block_tables"), (dict(block_tables=t(3 * B, d=i32)), SHAPE, "block_tables")]
WRONG = {
    "kvq_rope_write": PAGES + STATUS + [
        (dict(k=t(N, HKV + 1, DH)), SHAPE, "k must"), (dict(v=t(N + 1, HKV, DH)), SHAPE, "v must"), (dict(q_out=t(N, HQ, DH, d=f32)), ARG, "q_out"),
        (dict(q_out=t(N + 1, HQ, DH)), SHAPE, "q_out"), (dict(q=t(N, DH, HQ).transpose(1, 2)), SHAPE, "dense"),
        (dict(positions=t(N + 1, d=i32)), SHAPE, "positions"), (dict(positions=t(2, 3, N, d=i32)), SHAPE, "positions"),
        (dict(positions=t(N, d=i64)), ARG, "positions"), (dict(turns=t(32, d=i32)), ARG, "turns"), (dict(axis=t(31, d=u8)), SHAPE, "axis"),
        (dict(axis=t(32, d=i32)), ARG, "axis"), (dict(q_weight=t(DH + 1)), SHAPE, "q_weight"), (dict(k_weight=t(DH, d=f32)), ARG, "k_weight"),
        (dict(eps="small"), ARG, "eps"), (dict(slot_mapping=t(N, d=i32)), ARG, "slot_mapping"), (dict(slot_mapping=t(N - 1, d=i64)), SHAPE, "slot_mapping")],
    "kvq_tree_attn": PAGES + STATUS + LENS + [
        (dict(cu_q_lens=t(B, d=i32)), SHAPE, "cu_q_lens"), (dict(parents=t(N + 1, d=i32)), SHAPE, "parents"), (dict(parents=t(N, d=i64)), ARG, "parents"),
        (dict(seq_lens=t(B + 1, d=i32)), SHAPE, "seq_lens"), (dict(workspace=t(64, d=f32)), ARG, "workspace"), (dict(out=t(N, HQ, DH + 1)), SHAPE, "out"),
        (dict(q=t(HQ, N, DH).transpose(0, 1)), SHAPE, "contiguous"), (dict(flags="x"), ARG, "flags"), (dict(q_scale=t(1)), ARG, "q_scale")],
    "kvq_tree_commit": LIST + STATUS + LENS + [
        (dict(accepted=t(B + 1, 4, d=i32)), SHAPE, "accepted"), (dict(num_accepted=t(B, d=i64)), ARG, "num_accepted"),
        (dict(new_lens=t(B + 1, d=i32)), SHAPE, "new_lens"), (dict(cu_q_lens=t(B, d=i32)), SHAPE, "cu_q_lens")],
    "kvq_copy_pages": LIST + STATUS + [(dict(copies=t(3, 3, d=i32)), SHAPE, "copies"), (dict(copies=t(6, d=i32)), SHAPE, "copies")],
    "kvq_pages_init": TAKEN,
    "kvq_pages_alloc": TAKEN + STATUS + LENS + [(dict(old_lens=t(B + 1, d=i32)), SHAPE, "old_lens"), (dict(new_lens=t(B, d=i64)), ARG, "new_lens")],
    "kvq_pages_fork": TAKEN + STATUS + LENS + [
        (dict(out_tables=t(4, 4, d=i32)), SHAPE, "out_tables"), (dict(parents=t(3, d=i32)), SHAPE, "parents"),
        (dict(copies=t(4, d=i32)), SHAPE, "copies"), (dict(out_lens=t(5, d=i32)), SHAPE, "out_lens")],
}
WRONG["kvq_pages_free"] = WRONG["kvq_pages_alloc"]


@pytest.mark.parametrize("op,over,status,word", [(op, *c) for op in WRONG for c in WRONG[op]])
def test_binding_refusals(step, op, over, status, word):
    with pytest.raises(step.KvqError) as e:
        getattr(step, op)(**dict(arguments(op), **over))
    assert e.value.status == status and word in str(e.value)


@pytest.mark.parametrize("op", sorted(WRONG))
def test_binding_wants_cuda_tensors_and_all_arguments(step, op):
    a = arguments(op)
    for positional in (False, True):
        with pytest.raises(step.KvqError) as e:
            getattr(step, op)(*a.values()) if positional else getattr(step, op)(**a)
        assert e.value.status == ARG and "CUDA" in str(e.value)
    for call_ in (lambda: getattr(step, op)(), lambda: getattr(step, op)(*a.values(), other=3),
                  lambda: getattr(step, op)(**{k: v for k, v in list(a.items())[1:]}), lambda: getattr(step, op)(*[7] * len(a))):
        with pytest.raises((TypeError, step.KvqError)):
            call_()
