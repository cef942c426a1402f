"""Rotation of queries and keys by their positions, with an optional norm per
head: fa_qk_rope, its gradient and fa_qk_rope_append for torch.

q [num_tokens, H, d] and k, v [num_tokens, Hkv, d] are bf16 with packed heads;
rows may be strided (slices of a fused projection).  positions is int32
[num_tokens] (kv_plan's, or those of a packed batch), freqs what rope_freqs
makes once per model.  layout: FA_ROPE_HALF pairs value i of a head with
i + rotary_dim / 2, FA_ROPE_INTERLEAVED 2i with 2i + 1; values past rotary_dim
stay.  q_weight, k_weight ([d] bf16 or float32): the head is first divided by
sqrt(mean(x^2) + eps) and multiplied by the weight; None: it is not.  Nothing
waits for the GPU and every call can be captured into a CUDA graph.  Errors and
stream are those of the paged cache's calls (paged.py).
"""
from __future__ import annotations

import math

import torch

from . import FA_ERR_UNSUPPORTED, FabwdError, fa_last_error, lib, paged

FA_ROPE_HALF = 0
FA_ROPE_INTERLEAVED = 1
FA_WEIGHT_BF16 = 0
FA_WEIGHT_F32 = 1


def _host():
    return paged._native or paged._host()


def rope_freqs(rotary_dim: int, base: float = 10000.0, factor: float = 1.0, original_len: int = 0, low: float = 1.0,
               high: float = 32.0, inv_freq=None, device="cuda") -> torch.Tensor:
    """Frequencies of rotary_dim / 2 pairs, int64 [rotary_dim / 2] on device:
    theta_i = base^(-2i / rotary_dim) in turns per position times 2^64, with the
    53 significant bits of the float64 numbers they are computed in.

    For contexts longer than the trained one: factor alone divides every
    frequency (positions are interpolated).  With original_len, the trained
    length, only slow pairs are: with r = original_len * theta / (2 pi) turns over
    it, g = (r - low) / (high - low) clamped to [0, 1],
    theta' = g theta + (1 - g) theta / factor (by parts, after Peng et al., YaRN,
    2023, which also multiplies the outputs by mscale = 0.1 ln(factor) + 1: pass
    that to the calls).  A changed base is just another base.  inv_freq: the
    angles per position in radians (rotary_dim / 2 of them, float64 best) for
    any other rule; the factors then apply to these.

    Computed on the host in 64 bits; make it once, not per call."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and >= 0, got {rotary_dim}")
    if not (factor > 0 and math.isfinite(factor)):
        raise ValueError(f"factor must be positive and finite, got {factor}")
    if inv_freq is None:
        if not (base > 0 and math.isfinite(base)):
            raise ValueError(f"base must be positive and finite, got {base}")
        theta = [math.pow(base, -2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    else:
        theta = torch.as_tensor(inv_freq, dtype=torch.float64).detach().flatten().tolist()
        if len(theta) != rotary_dim // 2 or not all(map(math.isfinite, theta)):
            raise ValueError(f"inv_freq must hold rotary_dim / 2 = {rotary_dim // 2} finite values, got {len(theta)}")
    if original_len < 0 or (original_len and not low < high):
        raise ValueError(f"original_len must be >= 0 and low < high, got {original_len}, {low}, {high}")
    out = []
    for t in theta:
        if original_len:
            keep = min(1.0, max(0.0, (original_len * abs(t) / (2 * math.pi) - low) / (high - low)))
            t = keep * t + (1.0 - keep) * t / factor
        else:
            t = t / factor
        turns = t / (2 * math.pi)
        units = round(math.ldexp(turns - math.floor(turns), 64)) % (1 << 64)
        out.append(units - (1 << 64) if units >> 63 else units)
    return torch.tensor(out, dtype=torch.int64, device=device)


def fa_qk_rope(q, k, positions, freqs, q_out, k_out, layout: int = FA_ROPE_HALF, mscale: float = 1.0, q_weight=None,
               k_weight=None, eps: float = 1e-6, stream=None):
    """Fills q_out and k_out in place (q_out may be q, k_out k)."""
    _host().rope(q, k, positions, freqs, layout, mscale, q_weight, k_weight, eps, (q_out, k_out), stream)


def qk_rope(q, k, positions, freqs, layout: int = FA_ROPE_HALF, mscale: float = 1.0, q_weight=None, k_weight=None,
            eps: float = 1e-6, out=None, stream=None):
    """Normed (with a weight) and rotated (q, k); k or q may be None.  out:
    (q_out, k_out) to fill instead of new tensors, q and k themselves allowed.
    New ones are cut from one allocation like kv_plan's.  See fa_qk_rope in
    include/fabwd.h."""
    return _host().rope(q, k, positions, freqs, layout, mscale, q_weight, k_weight, eps, out, stream)


def fa_qk_rope_bwd_workspace_size(head_dim: int) -> int:
    n = lib().fa_qk_rope_bwd_workspace_size(head_dim)
    if n == 0:
        raise FabwdError(FA_ERR_UNSUPPORTED, fa_last_error())
    return int(n)


def fa_qk_rope_bwd(dq_out, dk_out, positions, freqs, dq, dk, dq_weight=None, dk_weight=None,
                   layout: int = FA_ROPE_HALF, mscale: float = 1.0, q=None, k=None, q_weight=None, k_weight=None,
                   eps: float = 1e-6, workspace=None, stream=None):
    """Fills dq, dk and, for tensors with a weight, dq_weight, dk_weight in place."""
    _host().rope_bwd(dq_out, dk_out, positions, freqs, layout, mscale, q_weight, k_weight, eps, q, k,
                     (dq, dk, dq_weight, dk_weight), workspace, stream)


def qk_rope_backward(dq_out, dk_out, positions, freqs, layout: int = FA_ROPE_HALF, mscale: float = 1.0, q=None, k=None,
                     q_weight=None, k_weight=None, eps: float = 1e-6, out=None, workspace=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) from the gradients dq_out, dk_out of
    qk_rope's outputs.  q, k: its inputs, needed where there is a weight.  The
    weights' gradients are float32, None without a weight.  out: such a tuple to
    fill (dq may be dq_out, dk dk_out).  workspace:
    fa_qk_rope_bwd_workspace_size() bytes to use instead of fresh ones (calls
    that may overlap need one each)."""
    return _host().rope_bwd(dq_out, dk_out, positions, freqs, layout, mscale, q_weight, k_weight, eps, q, k, out,
                            workspace, stream)


def fa_qk_rope_append(q, k, v, positions, freqs, k_cache, v_cache, slots, q_out, layout: int = FA_ROPE_HALF,
                      mscale: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6, k_scale=None, v_scale=None,
                      stream=None):
    """Fills q_out (which may be q) and the cache's slots in place."""
    _host().rope_append(q, k, v, positions, freqs, layout, mscale, q_weight, k_weight, eps, k_cache, v_cache, slots,
                        k_scale, v_scale, q_out, stream)


def qk_rope_append(q, k, v, positions, freqs, k_cache, v_cache, slots, layout: int = FA_ROPE_HALF, mscale: float = 1.0,
                   q_weight=None, k_weight=None, eps: float = 1e-6, k_scale=None, v_scale=None, out=None, stream=None):
    """qk_rope and kv_append in one pass: returns the rotated q; rotated keys
    and the values go into the cache at slots (kv_plan's; rows with slot -1 are
    skipped there)."""
    return _host().rope_append(q, k, v, positions, freqs, layout, mscale, q_weight, k_weight, eps, k_cache, v_cache,
                               slots, k_scale, v_scale, out, stream)
