"""Paged key/value cache: fa_kv_plan, fa_kv_append, fa_decode and fa_extend for
torch.

k_cache and v_cache are [num_pages, page_size, Hkv, d] tensors, bf16 or
float8_e4m3fn, in any strided layout whose last dimension is contiguous
(``cache.permute(0, 2, 1, 3)`` of a [num_pages, Hkv, page_size, d] tensor,
``cache[:, 0]`` of a [num_pages, 2, page_size, Hkv, d] one), the same for
both.  Unlike the packed entry points these take everything from device
tensors: nothing waits for the GPU and every call can be captured into a
CUDA graph.  What the C layer cannot see (types, shapes, strides, devices)
is checked in the host extension (csrc/paged_host.cpp) and raises
ValueError; FabwdError comes from the C layer.

stream: a torch.cuda.Stream of the tensors' device to run on (and to
allocate outputs on) instead of the current one.  The caller orders it after
what writes the inputs; their memory is kept until the stream is done.
"""
from __future__ import annotations

import os
from typing import NamedTuple

import torch

from . import FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FabwdError, fa_last_error, lib

FA_KV_BF16 = 0
FA_KV_E4M3 = 1

_native = None


def _host():
    """The host extension, built beside libfabwd.so (no fallback)."""
    global _native
    if _native is None:
        lib()   # says how to build if nothing is built
        if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_paged_host.so")):
            raise RuntimeError("_paged_host.so is missing: build it with python attention_backward_sm_gb300/build.py")
        from . import _paged_host
        _native = _paged_host
    return _native


class KvPlan(NamedTuple):
    """What kv_plan returns: slots int64 and positions int32 per new token,
    cu_new int32 [batch + 1], seq_lens int32 [batch] with the new tokens
    counted, free_next int32 [1].  They are cut from one allocation: keeping
    one keeps all (as does record_stream), and torch.save of one writes all
    unless it is cloned.  fa_kv_plan fills tensors of your own."""
    slots: torch.Tensor
    positions: torch.Tensor
    cu_new: torch.Tensor
    seq_lens: torch.Tensor
    free_next: torch.Tensor


def fa_kv_plan(block_table, seq_lens, new_lens, free_pages, page_size: int, slots, positions, cu_new, seq_lens_out,
               free_next, free_start=None, stream=None):
    """Fills slots (int64), positions, cu_new, seq_lens_out, free_next and the
    new entries of block_table in place."""
    (_native or _host()).plan(block_table, seq_lens, new_lens, free_pages, page_size, slots.numel(), free_start,
                              (slots, positions, cu_new, seq_lens_out, free_next), stream)


def kv_plan(block_table, seq_lens, new_lens, free_pages, page_size: int, num_tokens: int, free_start=None,
            stream=None) -> KvPlan:
    """Gives num_tokens new tokens (new_lens per request, padded if there are
    fewer) their slots and positions, entering the pages they need from
    free_pages into block_table.  See fa_kv_plan in include/fabwd.h."""
    return KvPlan._make((_native or _host()).plan(block_table, seq_lens, new_lens, free_pages, page_size, num_tokens,
                                                  free_start, None, stream))


def fa_kv_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, stream=None):
    """Writes rows k, v [num_tokens, Hkv, d] (rows may be strided) to slots."""
    (_native or _host()).append(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream)


def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, stream=None):
    """Writes the rows of k and v [num_tokens, Hkv, d] into the cache at
    slots (kv_plan's); rows with slot -1 are skipped."""
    (_native or _host()).append(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream)


def fa_decode_workspace_size(batch: int, heads: int, heads_kv: int, head_dim: int) -> int:
    n = lib().fa_decode_workspace_size(batch, heads, heads_kv, head_dim)
    err = fa_last_error()
    if err:   # the size function gives no code
        raise FabwdError(FA_ERR_UNSUPPORTED if err.startswith("head_dim") else FA_ERR_INVALID_ARG, err)
    return int(n)


def fa_decode(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale: float, window: int = 0, k_scale=None,
              v_scale=None, workspace=None, stream=None):
    """Fills o (bf16, contiguous) and lse (fp32, or None) in place."""
    (_native or _host()).decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, k_scale, v_scale, (o, lse),
                                workspace, stream)


def decode(q, k_cache, v_cache, block_table, seq_lens, scale: float, window: int = 0, k_scale=None, v_scale=None,
           out=None, workspace=None, stream=None):
    """Attention of one new token per request, q [batch, H, d], over the
    cache; returns (o, lse), cut from one allocation like kv_plan's.  out:
    (o, lse) to fill instead of new tensors (lse may be None).  workspace: fa_decode_workspace_size() bytes to use
    instead of fresh ones (calls that may overlap need one each)."""
    return (_native or _host()).decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, k_scale, v_scale, out,
                                       workspace, stream)


def fa_extend_workspace_size(head_dim: int) -> int:
    n = lib().fa_extend_workspace_size(head_dim)
    if n == 0:
        raise FabwdError(FA_ERR_UNSUPPORTED, fa_last_error())
    return int(n)


def fa_extend(q, k_cache, v_cache, block_table, seq_lens, cu_new, o, lse, scale: float, window: int = 0, k_scale=None,
              v_scale=None, workspace=None, stream=None):
    """Fills o (bf16, contiguous) and lse (fp32, or None) in place."""
    (_native or _host()).extend(q, k_cache, v_cache, block_table, seq_lens, cu_new, scale, window, k_scale, v_scale,
                                (o, lse), workspace, stream)


def extend(q, k_cache, v_cache, block_table, seq_lens, cu_new, scale: float, window: int = 0, k_scale=None,
           v_scale=None, out=None, workspace=None, stream=None):
    """Attention of the new tokens q [num_tokens, H, d] over the cache, causal
    within each request; seq_lens and cu_new are kv_plan's.  Returns (o, lse),
    cut from one allocation like kv_plan's.  out: (o, lse) to fill instead of new
    tensors (lse may be None).  workspace: fa_extend_workspace_size() bytes to use
    instead of fresh ones (calls that may overlap need one each)."""
    return (_native or _host()).extend(q, k_cache, v_cache, block_table, seq_lens, cu_new, scale, window, k_scale,
                                       v_scale, out, workspace, stream)
