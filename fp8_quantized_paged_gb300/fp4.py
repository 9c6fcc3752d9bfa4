"""Binding of the microscaled 4-bit cache (``include/kvq_fp4.h``).

The functions carry the C names and are also found in the package itself.
Caches are uint8 ``[num_blocks][Hkv][9 * head_dim]`` (``new_fp4_cache``);
scales are fp32 ``[1]`` or ``[Hkv]``.  Tensors are checked here for what the C
ABI cannot see from a pointer: element type, dense layout, length and device.
"""
from __future__ import annotations

import ctypes

import torch

from . import BLOCK_SIZE, KVQ_ERR_ARG, KVQ_ERR_SHAPE, KVQ_OK, KvqError, _i32, _i64, _stream, _sz, _vp, lib

SIGNATURES = {
    "kvq_fp4_write": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp, _i64, _i32, _vp, _i32,
                             _vp, _i32, _i32, _vp, _vp]),
    "kvq_fp4_read": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _i32, _i64, _vp,
                            _i32, _vp, _i32, _i32, _vp, _vp, _i64, _vp, _vp]),
    "kvq_fp4_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "kvq_fp4_decode_attn": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i64,
                                   _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp, _sz, _vp,
                                   _vp, _vp]),
    "kvq_fp4_prefill_attn": (_i32, [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                    _i32, _i32, _i64, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                    _vp, _sz, _vp, _vp, _vp]),
}

_lib = lib()
for _name, (_res, _args) in SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args

_BF16, _U8, _I32, _I64, _F32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32


def _fail(where, text, status=KVQ_ERR_SHAPE):
    raise KvqError(status, f"{where}: {text}")


def _device(where, t):
    """The device of a call: that of its first tensor, which has to be CUDA's
    current one (the kernels run there)."""
    dev = t.get_device()
    if dev < 0:
        _fail(where, "tensors must be CUDA tensors", KVQ_ERR_ARG)
    if dev != torch.cuda.current_device():
        _fail(where, f"tensors are on cuda:{dev}, not on the current device", KVQ_ERR_ARG)
    return dev


def _need(where, dev, t, name, dtype, shape=None):
    """t: a dense tensor of this type, shape (None: any) and device."""
    if t.dtype is not dtype:
        _fail(where, f"{name} must be {dtype}, got {t.dtype}", KVQ_ERR_ARG)
    if t.get_device() != dev:
        _fail(where, f"{name} must be on the device of the other tensors", KVQ_ERR_ARG)
    if not t.is_contiguous():
        _fail(where, f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        _fail(where, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _need_rows(where, dev, t, name, shape):
    """t: bf16 rows [n][heads][head_dim], dense but for the distance of consecutive
    rows.  Returns (pointer, that distance)."""
    if t.dtype is not _BF16:
        _fail(where, f"{name} must be {_BF16}, got {t.dtype}", KVQ_ERR_ARG)
    if t.get_device() != dev:
        _fail(where, f"{name} must be on the device of the other tensors", KVQ_ERR_ARG)
    if t.shape != shape:
        _fail(where, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    n, heads, dh = shape
    s0, s1, s2 = t.stride()
    if (s1 != dh and heads > 1) or s2 != 1:
        _fail(where, f"{name} must be dense within a row")
    return t.data_ptr(), (s0 if n > 1 else heads * dh)


def _need_status(where, dev, t):
    if t is None:
        return None
    if t.element_size() != 4 or t.numel() < 1:
        _fail(where, "dev_status must hold a 32-bit word", KVQ_ERR_ARG)
    if t.get_device() != dev:
        _fail(where, "dev_status must be on the device of the other tensors", KVQ_ERR_ARG)
    return t.data_ptr()


def _need_caches(where, dev, k_cache, v_cache, head_dim=None):
    if k_cache.dim() != 3:
        _fail(where, "caches must have shape [num_blocks][Hkv][9 * head_dim]")
    shape = k_cache.shape
    if shape[2] % 9 or (head_dim is not None and shape[2] != 9 * head_dim):
        _fail(where, f"a cache page of {shape[2]} bytes is not 9 * head_dim")
    return (_need(where, dev, k_cache, "k_cache", _U8), _need(where, dev, v_cache, "v_cache", _U8, shape),
            shape[0], shape[1], shape[2] // 9)


def kvq_fp4_write(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, scale_granularity,
                  dev_status=None, stream=None) -> None:
    """Quantize-and-scatter: k, v bf16 [N][Hkv][dh] (rows may lie further apart
    than Hkv * dh), slot_mapping int64 [N] (negative: skipped)."""
    where = "kvq_fp4_write"
    dev = _device(where, k)
    n, hkv, dh = shape = k.shape
    kp, ks = _need_rows(where, dev, k, "k", shape)
    vp, vs = _need_rows(where, dev, v, "v", shape)
    if ks != vs:
        _fail(where, "k and v must have the same row distance")
    kc, vc, nb, chkv, _ = _need_caches(where, dev, k_cache, v_cache, dh)
    if chkv != hkv:
        _fail(where, f"the caches hold {chkv} KV heads, k and v {hkv}")
    st = _lib.kvq_fp4_write(
        kp, vp, ks, _need(where, dev, slot_mapping, "slot_mapping", _I64, (n,)), n, hkv, dh, kc, vc,
        nb, BLOCK_SIZE, _need(where, dev, k_scale, "k_scale", _F32), k_scale.numel(),
        _need(where, dev, v_scale, "v_scale", _F32), v_scale.numel(), scale_granularity,
        _need_status(where, dev, dev_status), _stream(stream))
    if st != KVQ_OK:
        raise KvqError(st, where)


def kvq_fp4_read(k_cache, v_cache, block_tables, starts, cu_lens, k_scale, v_scale,
                 scale_granularity, k_out, v_out, dev_status=None, stream=None) -> None:
    """Gather tokens back to bf16: rows cu_lens[b] .. cu_lens[b + 1] of k_out and
    v_out [num_rows][Hkv][dh] are the tokens of sequence b from starts[b] on
    (starts None: from its first).  cu_lens int32 [B + 1]; rows from cu_lens[B]
    on are left as they were."""
    where = "kvq_fp4_read"
    dev = _device(where, k_cache)
    kc, vc, nb, hkv, dh = _need_caches(where, dev, k_cache, v_cache)
    n = k_out.shape[0]
    kp, ks = _need_rows(where, dev, k_out, "k_out", (n, hkv, dh))
    vp, vs = _need_rows(where, dev, v_out, "v_out", (n, hkv, dh))
    if ks != vs:
        _fail(where, "k_out and v_out must have the same row distance")
    B, mb = block_tables.shape
    st = _lib.kvq_fp4_read(
        kc, vc, nb, BLOCK_SIZE, hkv, dh, _need(where, dev, block_tables, "block_tables", _I32), mb,
        None if starts is None else _need(where, dev, starts, "starts", _I32, (B,)),
        _need(where, dev, cu_lens, "cu_lens", _I32, (B + 1,)), B, n,
        _need(where, dev, k_scale, "k_scale", _F32), k_scale.numel(),
        _need(where, dev, v_scale, "v_scale", _F32), v_scale.numel(), scale_granularity, kp, vp, ks,
        _need_status(where, dev, dev_status), _stream(stream))
    if st != KVQ_OK:
        raise KvqError(st, where)


def kvq_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, num_sms=0) -> int:
    return int(_lib.kvq_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, num_sms))


def kvq_fp4_decode_attn(q, k_cache, v_cache, block_tables, seq_lens, k_scale, v_scale,
                        scale_granularity, sliding_window, num_sinks, workspace, out,
                        dev_status=None, stream=None) -> None:
    """Decode attention: q bf16 [B][Hq][dh] -> out; each query sees its sequence's
    last sliding_window tokens (0: all) and its first num_sinks."""
    where = "kvq_fp4_decode_attn"
    dev = _device(where, q)
    B, hq, dh = shape = q.shape
    kc, vc, nb, hkv, _ = _need_caches(where, dev, k_cache, v_cache, dh)
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        _fail(where, f"block_tables must have shape [{B}][max_blocks_per_seq]")
    st = _lib.kvq_fp4_decode_attn(
        _need(where, dev, q, "q", _BF16), kc, vc,
        _need(where, dev, block_tables, "block_tables", _I32), block_tables.shape[1],
        _need(where, dev, seq_lens, "seq_lens", _I32, (B,)), B, hq, hkv, dh, nb, BLOCK_SIZE,
        _need(where, dev, k_scale, "k_scale", _F32), k_scale.numel(),
        _need(where, dev, v_scale, "v_scale", _F32), v_scale.numel(), scale_granularity,
        sliding_window, num_sinks, _need(where, dev, workspace, "workspace", _U8), workspace.numel(),
        _need(where, dev, out, "out", _BF16, shape), _need_status(where, dev, dev_status),
        _stream(stream))
    if st != KVQ_OK:
        raise KvqError(st, where)


def kvq_fp4_prefill_attn(q, cu_q_lens, max_q_len, k_cache, v_cache, block_tables, seq_lens, k_scale,
                         v_scale, scale_granularity, sliding_window, num_sinks, workspace, out,
                         dev_status=None, stream=None) -> None:
    """Prefill attention: q bf16 [total_q][Hq][dh], cu_q_lens int32 [B + 1] (device),
    max_q_len a host bound of the chunks' lengths; a chunk is its sequence's
    last tokens, each of which sees what kvq_fp4_decode_attn shows it."""
    where = "kvq_fp4_prefill_attn"
    dev = _device(where, q)
    n, hq, dh = shape = q.shape
    kc, vc, nb, hkv, _ = _need_caches(where, dev, k_cache, v_cache, dh)
    B = seq_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        _fail(where, f"block_tables must have shape [{B}][max_blocks_per_seq]")
    st = _lib.kvq_fp4_prefill_attn(
        _need(where, dev, q, "q", _BF16), _need(where, dev, cu_q_lens, "cu_q_lens", _I32, (B + 1,)),
        n, max_q_len, kc, vc, _need(where, dev, block_tables, "block_tables", _I32),
        block_tables.shape[1], _need(where, dev, seq_lens, "seq_lens", _I32, (B,)), B, hq, hkv, dh,
        nb, BLOCK_SIZE, _need(where, dev, k_scale, "k_scale", _F32), k_scale.numel(),
        _need(where, dev, v_scale, "v_scale", _F32), v_scale.numel(), scale_granularity,
        sliding_window, num_sinks, _need(where, dev, workspace, "workspace", _U8), workspace.numel(),
        _need(where, dev, out, "out", _BF16, shape), _need_status(where, dev, dev_status),
        _stream(stream))
    if st != KVQ_OK:
        raise KvqError(st, where)


# --------------------------------------------------------------------------
# allocation helpers (torch memory; no compute)
# --------------------------------------------------------------------------

def new_fp4_cache(num_blocks, num_kv_heads, head_dim, device="cuda"):
    """One tensor's pages, zero: a page never written reads as zeros."""
    return torch.zeros((num_blocks, num_kv_heads, 9 * head_dim), dtype=_U8, device=device)


def new_fp4_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, device="cuda"):
    """A workspace for both attentions, zero-filled (its counters must start at zero)."""
    n = kvq_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise KvqError(KVQ_ERR_ARG, "kvq_fp4_workspace_size")
    return torch.zeros(n, dtype=_U8, device=device)
