"""Plain definition of the paged key/value cache operators (float64 numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package: plan, append and
single-token attention, one request (and one key/value head) at a time.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64


def plan(table, seq_lens, new_lens, free_pages, page_size: int, num_tokens: int, free_start: int = 0):
    """Returns (table, slots, positions, cu_new, seq_lens, free_next), token
    by token: a token at position p sits in page p // page_size of its
    request; a page the request does not hold yet is the next free one."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    slots = np.full(num_tokens, -1, dtype=np.int64)
    positions = np.zeros(num_tokens, dtype=np.int64)
    cu, after, nxt, at = [0], [], int(free_start), 0
    for b, (s, n) in enumerate(zip(seq_lens, new_lens)):
        s, n = max(int(s), 0), max(int(n), 0)
        for p in range(s, s + n):
            j = p // page_size
            if j < width and p % page_size == 0:
                table[b, j] = free_pages[nxt] if nxt < len(free_pages) else -1
                nxt += 1
            if at < num_tokens:
                positions[at] = p
                if j < width and table[b, j] >= 0:
                    slots[at] = table[b, j] * page_size + p % page_size
            at += 1
        cu.append(at)
        after.append(s + n)
    return table, slots, positions, np.array(cu), np.array(after), nxt


def e4m3(x) -> np.ndarray:
    """Nearest value with 3 fraction bits and exponents -6..8 (steps of 2^-9
    below 2^-6), ties to even, saturating at +-448; NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    power = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = np.exp2(power - 3)
    r = np.minimum(np.rint(a / step) * step, 448.0)
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def decode(q, k_cache, v_cache, table, seq_lens, scale: float, window: int = 0, k_scale=None, v_scale=None):
    """(o, lse, p_abs_v, x_abs) of single-token attention over the cache:
    o [B, H, d], lse [B, H], and for error bounds p_abs_v = sum_j p_j |v_j|
    [B, H, d] and x_abs = max_j scale * sum_c |q_c k_jc| [B, H]."""
    q, k_cache, v_cache = _f64(q), _f64(k_cache), _f64(v_cache)
    table, seq_lens = np.asarray(table), np.asarray(seq_lens)
    B, H, d = q.shape
    pages, ps, Hkv, _ = k_cache.shape
    ks = np.ones(Hkv) if k_scale is None else _f64(k_scale)
    vs = np.ones(Hkv) if v_scale is None else _f64(v_scale)
    o, pv = np.zeros((B, H, d)), np.zeros((B, H, d))
    lse, xa = np.full((B, H), -np.inf), np.zeros((B, H))
    for b in range(B):
        n = min(max(int(seq_lens[b]), 0), table.shape[1] * ps)
        j = np.arange(max(0, n - window) if window else 0, n)
        page = table[b][j // ps] if n else j
        ok = (page >= 0) & (page < pages)
        j, page = j[ok], page[ok]
        if len(j) == 0:
            continue
        for h in range(H):
            hk = h // (H // Hkv)
            k = k_cache[page, j % ps, hk] * ks[hk]
            v = v_cache[page, j % ps, hk] * vs[hk]
            x = scale * (k @ q[b, h])
            e = np.exp(x - x.max())
            p = e / e.sum()
            o[b, h], pv[b, h] = p @ v, p @ np.abs(v)
            lse[b, h] = x.max() + np.log(e.sum())
            xa[b, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
    return o, lse, pv, xa
