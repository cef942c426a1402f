"""Paged key/value cache: binding of fa_kv_plan, fa_kv_append and fa_decode.

k_cache and v_cache are [num_pages, page_size, Hkv, d] tensors, bf16 or
float8_e4m3fn, in any strided layout whose last dimension is contiguous
(``cache.permute(0, 2, 1, 3)`` of a [num_pages, Hkv, page_size, d] tensor,
``cache[:, 0]`` of a [num_pages, 2, page_size, Hkv, d] one), the same for
both.  Unlike the packed entry points these take everything from device
tensors: nothing waits for the GPU and every call can be captured into a
CUDA graph.  What the C layer cannot see (types, shapes, strides, devices)
is checked here and raises ValueError; FabwdError comes from the C layer.
"""
from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from . import FA_ERR_INVALID_ARG, FabwdError, _check, _ptr, _raw_stream, fa_last_error, lib

FA_KV_BF16 = 0
FA_KV_E4M3 = 1

_KV_TYPES = {torch.bfloat16: FA_KV_BF16, torch.float8_e4m3fn: FA_KV_E4M3}


def _launch(fn, device, stream, *args):
    """fn(*args, stream) on the tensors' device, whichever device is current."""
    if stream is None:
        raw = _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        _check(fn(*args, raw or None))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, raw or None))


def _same_device(device, **tensors):
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, got {device}")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the others on {device}")


def _vector(name, t, dtype, n=None):
    if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        size = "" if n is None else f" of {n}"
        raise ValueError(f"{name} must be a contiguous {dtype} vector{size}, got {t.dtype} {tuple(t.shape)}")


def _row_stride(name, t, n, heads, dim):
    """Elements from one row of a [n, heads, dim] bf16 tensor to the next."""
    if t.dtype != torch.bfloat16 or tuple(t.shape) != (n, heads, dim):
        raise ValueError(f"{name} must be bfloat16 {(n, heads, dim)}, got {t.dtype} {tuple(t.shape)}")
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != dim):
        raise ValueError(f"{name} must have its heads packed in each row, got strides {st}")
    return st[0] if n > 1 else heads * dim


def _cache_args(k_cache, v_cache, k_scale, v_scale):
    """Shape of the cache and its C arguments up to page_size."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape [num_pages, page_size, Hkv, d], got "
                         f"{tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
    kind = _KV_TYPES.get(k_cache.dtype)
    if kind is None or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must both be bfloat16 or both float8_e4m3fn, got "
                         f"{k_cache.dtype} and {v_cache.dtype}")
    st = k_cache.stride()
    if st[3] != 1 or v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must have the same strides, the last 1, got "
                         f"{st} and {v_cache.stride()}")
    pages, page_size, heads_kv, dim = k_cache.shape
    if k_scale is not None:
        _vector("k_scale", k_scale, torch.float32, heads_kv)
    if v_scale is not None:
        _vector("v_scale", v_scale, torch.float32, heads_kv)
    return (pages, page_size, heads_kv, dim), (_ptr(k_cache), _ptr(v_cache), kind, _ptr(k_scale), _ptr(v_scale),
                                               st[0], st[1], st[2], pages, page_size)


def _table_args(block_table):
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError(f"block_table must be int32 [batch, max_pages], got {block_table.dtype} "
                         f"{tuple(block_table.shape)}")
    batch, width = block_table.shape
    st = block_table.stride()
    if width > 1 and st[1] != 1:
        raise ValueError(f"block_table must have contiguous rows, got strides {st}")
    return batch, (_ptr(block_table), st[0] if batch > 1 else width, width)


def fa_kv_plan(block_table, seq_lens, new_lens, free_pages, page_size: int, slots, positions, cu_new, seq_lens_out,
               free_next, free_start=None, stream=None):
    """Fills slots (int64), positions, cu_new, seq_lens_out, free_next and the
    new entries of block_table in place."""
    batch, table = _table_args(block_table)
    _vector("seq_lens", seq_lens, torch.int32, batch)
    _vector("new_lens", new_lens, torch.int32, batch)
    _vector("free_pages", free_pages, torch.int32)
    _vector("slots", slots, torch.int64)
    _vector("positions", positions, torch.int32, slots.shape[0])
    _vector("cu_new", cu_new, torch.int32, batch + 1)
    _vector("seq_lens_out", seq_lens_out, torch.int32, batch)
    _vector("free_next", free_next, torch.int32, 1)
    if free_start is not None:
        _vector("free_start", free_start, torch.int32, 1)
    device = block_table.device
    _same_device(device, seq_lens=seq_lens, new_lens=new_lens, free_pages=free_pages, slots=slots,
                 positions=positions, cu_new=cu_new, seq_lens_out=seq_lens_out, free_next=free_next,
                 free_start=free_start)
    _launch(lib().fa_kv_plan, device, stream, *table, _ptr(seq_lens), _ptr(new_lens), _ptr(free_pages),
            free_pages.shape[0], _ptr(free_start), int(page_size), batch, slots.shape[0], _ptr(slots),
            _ptr(positions), _ptr(cu_new), _ptr(seq_lens_out), _ptr(free_next))


def fa_kv_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, stream=None):
    """Writes rows k, v [num_tokens, Hkv, d] (rows may be strided) to slots."""
    (_, _, heads_kv, dim), cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    _vector("slots", slots, torch.int64)
    n = slots.shape[0]
    k_stride = _row_stride("k", k, n, heads_kv, dim)
    v_stride = _row_stride("v", v, n, heads_kv, dim)
    device = k_cache.device
    _same_device(device, k=k, v=v, slots=slots, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
    _launch(lib().fa_kv_append, device, stream, _ptr(k), _ptr(v), k_stride, v_stride, _ptr(slots), n, *cache,
            heads_kv, dim)


@functools.lru_cache(maxsize=None)
def fa_decode_workspace_size(batch: int, heads: int, heads_kv: int, head_dim: int) -> int:
    n = lib().fa_decode_workspace_size(batch, heads, heads_kv, head_dim)
    err = fa_last_error()
    if err:
        raise FabwdError(FA_ERR_INVALID_ARG, err)
    return int(n)


def fa_decode(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale: float, window: int = 0, k_scale=None,
              v_scale=None, workspace=None, stream=None):
    """Fills o (bf16, contiguous) and lse (fp32, or None) in place."""
    (_, _, heads_kv, dim), cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    batch, table = _table_args(block_table)
    if q.dim() != 3:
        raise ValueError(f"q must be [batch, H, d], got {tuple(q.shape)}")
    heads = q.shape[1]
    q_stride = _row_stride("q", q, batch, heads, dim)
    _row_stride("o", o, batch, heads, dim)
    if not o.is_contiguous():
        raise ValueError("o must be contiguous")
    _vector("seq_lens", seq_lens, torch.int32, batch)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (batch, heads)
                            or not lse.is_contiguous()):
        raise ValueError(f"lse must be contiguous float32 {(batch, heads)}, got {lse.dtype} {tuple(lse.shape)}")
    device = q.device
    _same_device(device, k_cache=k_cache, v_cache=v_cache, block_table=block_table, seq_lens=seq_lens, o=o, lse=lse,
                 k_scale=k_scale, v_scale=v_scale, workspace=workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch(lib().fa_decode, device, stream, _ptr(q), q_stride, *cache, *table, _ptr(seq_lens), batch, heads,
            heads_kv, dim, int(window), float(scale), _ptr(o), _ptr(lse), _ptr(workspace), ws_bytes)


class KvPlan(NamedTuple):
    """What kv_plan returns: slots int64 and positions int32 per new token,
    cu_new int32 [batch + 1], seq_lens int32 [batch] with the new tokens
    counted, free_next int32 [1]."""
    slots: torch.Tensor
    positions: torch.Tensor
    cu_new: torch.Tensor
    seq_lens: torch.Tensor
    free_next: torch.Tensor


def kv_plan(block_table, seq_lens, new_lens, free_pages, page_size: int, num_tokens: int, free_start=None,
            stream=None) -> KvPlan:
    """Gives num_tokens new tokens (new_lens per request, padded if there are
    fewer) their slots and positions, entering the pages they need from
    free_pages into block_table.  See fa_kv_plan in include/fabwd.h."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_plan(block_table, seq_lens, new_lens, free_pages, page_size, num_tokens, free_start)
    device = block_table.device
    batch = block_table.shape[0]
    new = block_table.new_empty
    out = KvPlan(torch.empty(num_tokens, dtype=torch.int64, device=device), new(num_tokens), new(batch + 1),
                 new(batch), new(1))
    fa_kv_plan(block_table, seq_lens, new_lens, free_pages, page_size, *out, free_start=free_start)
    return out


def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, stream=None):
    """Writes the rows of k and v [num_tokens, Hkv, d] into the cache at
    slots (kv_plan's); rows with slot -1 are skipped."""
    fa_kv_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream)


def decode(q, k_cache, v_cache, block_table, seq_lens, scale: float, window: int = 0, k_scale=None, v_scale=None,
           out=None, workspace=None, stream=None):
    """Attention of one new token per request, q [batch, H, d], over the
    cache; returns (o, lse).  out: (o, lse) to fill instead of new tensors.
    workspace: fa_decode_workspace_size() bytes to use instead of fresh ones
    (calls that may overlap need one each)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, k_scale, v_scale, out, workspace)
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError(f"q must be [batch, H, d] and the caches [num_pages, page_size, Hkv, d], got "
                         f"{tuple(q.shape)} and {tuple(k_cache.shape)}")
    batch, heads, dim = q.shape
    device = q.device
    if out is None:
        out = (torch.empty((batch, heads, dim), dtype=q.dtype, device=device),
               torch.empty((batch, heads), dtype=torch.float32, device=device))
    o, lse = out
    if workspace is None:
        n = fa_decode_workspace_size(batch, heads, k_cache.shape[2], dim)
        if n > 0:
            workspace = torch.empty(n, dtype=torch.uint8, device=device)
    fa_decode(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale, window, k_scale, v_scale, workspace)
    return o, lse
