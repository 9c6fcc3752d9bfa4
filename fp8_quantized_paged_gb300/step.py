"""Binding of the operators around a serving step (``include/kvq_step.h``).

The functions carry the C names and are also found in the package itself.  The
compute entry points are native (``csrc/step_binding.cpp``) and check what the C
ABI cannot see from a pointer, as those of ``fp4`` do.  Cache lists may mix the
FP8, bf16, scale and 4-bit caches of ``new_cache``, ``new_scale_cache`` and
``new_fp4_cache``.
"""
from __future__ import annotations

import math

import torch

from . import KVQ_ERR_ARG, KvqError, _i32, _sz, lib
from .fp4 import _native

KVQ_DEV_NO_PAGES, KVQ_DEV_BAD_TREE = 64, 128
KVQ_TREE_MAX_NODES = 256
KVQ_POOL_HEADER = 4

kvq_rope_write = _native.kvq_rope_write
kvq_tree_attn = _native.kvq_tree_attn
kvq_tree_commit = _native.kvq_tree_commit
kvq_copy_pages = _native.kvq_copy_pages
kvq_pages_init = _native.kvq_pages_init
kvq_pages_alloc = _native.kvq_pages_alloc
kvq_pages_free = _native.kvq_pages_free
kvq_pages_fork = _native.kvq_pages_fork

_size = lib().kvq_tree_workspace_size
_size.restype, _size.argtypes = _sz, [_i32] * 4


def kvq_tree_workspace_size(num_q_heads, num_kv_heads, head_dim, num_sms=0) -> int:
    return int(_size(num_q_heads, num_kv_heads, head_dim, num_sms))


# --------------------------------------------------------------------------
# allocation helpers (torch memory; no compute)
# --------------------------------------------------------------------------

def new_tree_workspace(num_q_heads, num_kv_heads, head_dim, device="cuda"):
    """A workspace of kvq_tree_attn; what it holds means nothing."""
    n = kvq_tree_workspace_size(num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise KvqError(KVQ_ERR_ARG, "kvq_tree_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def new_page_pool(num_blocks, device="cuda"):
    """A pool of num_blocks pages, all free: int32 words, of which [1] counts the free pages
    and [4:4 + num_blocks] each page's holders."""
    if not 0 < num_blocks <= 1 << 24:
        raise KvqError(KVQ_ERR_ARG, "new_page_pool")
    pool = torch.zeros(KVQ_POOL_HEADER + num_blocks + (num_blocks + 31) // 32, dtype=torch.int32)
    pool[1] = num_blocks
    pool[KVQ_POOL_HEADER + num_blocks:] = -1
    if num_blocks % 32:
        pool[-1] = (1 << num_blocks % 32) - 1
    return pool.to(device)


def rope_turns(inv_freq, device="cuda"):
    """The turns of kvq_rope_write for frequencies of inv_freq radians a position (numbers, or a
    tensor; whatever scaling a model has is applied to them before): round(2^64 f / 2 pi) mod 2^64."""
    f = inv_freq.double().tolist() if isinstance(inv_freq, torch.Tensor) else [float(x) for x in inv_freq]
    t = [round(x / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for x in f]
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in t], dtype=torch.int64, device=device)
