"""Binding of the microscaled 4-bit cache (``include/kvq_fp4.h``).

The functions carry the C names and are also found in the package itself.
Caches are uint8 ``[num_blocks][Hkv][9 * head_dim]`` (``new_fp4_cache``);
scales are fp32 ``[1]`` or ``[Hkv]``.  The compute entry points are native
(``csrc/fp4_binding.cpp``): they check what the C ABI cannot see from a pointer
(element type, dense layout, length, one device, the current one), pass the
current stream unless given another, and raise ``KvqError``.
"""
from __future__ import annotations

import importlib.util
import os

import torch

from . import KVQ_ERR_ARG, LIB_PATH, KvqError, _i32, _sz, lib

NATIVE_PATH = os.path.join(os.path.dirname(LIB_PATH), "_kvq_fp4.so")


def _load_native():
    if not os.path.exists(NATIVE_PATH):
        raise ImportError(f"the 4-bit cache's binding is not built ({NATIVE_PATH} missing); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    spec = importlib.util.spec_from_file_location("_kvq_fp4", NATIVE_PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.bind(LIB_PATH, KvqError)
    return m


_native = _load_native()
kvq_fp4_write = _native.kvq_fp4_write
kvq_fp4_read = _native.kvq_fp4_read
kvq_fp4_decode_attn = _native.kvq_fp4_decode_attn
kvq_fp4_prefill_attn = _native.kvq_fp4_prefill_attn

_size = lib().kvq_fp4_workspace_size
_size.restype, _size.argtypes = _sz, [_i32] * 5


def kvq_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, num_sms=0) -> int:
    return int(_size(num_seqs, num_q_heads, num_kv_heads, head_dim, num_sms))


# --------------------------------------------------------------------------
# allocation helpers (torch memory; no compute)
# --------------------------------------------------------------------------

def new_fp4_cache(num_blocks, num_kv_heads, head_dim, device="cuda"):
    """One tensor's pages, zero: a page never written reads as zeros."""
    return torch.zeros((num_blocks, num_kv_heads, 9 * head_dim), dtype=torch.uint8, device=device)


def new_fp4_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, device="cuda"):
    """A workspace for both attentions, zero-filled (its counters must start at zero)."""
    n = kvq_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise KvqError(KVQ_ERR_ARG, "kvq_fp4_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)
