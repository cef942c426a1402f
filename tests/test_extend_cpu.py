"""Attention of several new tokens over the paged cache without a GPU: the
oracle's pins and the refusals of the C entry point (before anything touches the
device)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import oracle
from oracle import paged


@pytest.fixture(scope="module")
def lib():
    from attention_backward_sm_gb300 import build
    build.build()
    from attention_backward_sm_gb300 import _lib
    return _lib.load()


@pytest.mark.parametrize("window", [0, 3])
def test_a_chunk_is_the_end_of_the_forward(window):
    """Over a permuted paged copy of packed K, V the new tokens' rows are the
    last rows of the causal forward."""
    rng = np.random.default_rng(3)
    H, Hkv, d, ps, lens, new = 4, 2, 8, 4, [9, 4, 11], [3, 4, 0]
    k_cache, v_cache = rng.normal(size=(2, 12, ps, Hkv, d))
    table = rng.permutation(12)[:9].reshape(3, 3)
    q = rng.normal(size=(9, H, d))
    o, lse, _, _, n = paged.extend(q, k_cache, v_cache, table, lens, [0, 3, 7, 7], 0.3, window)
    for b, (s, m) in enumerate(zip(lens, new)):
        k, v = (c[table[b]].reshape(-1, Hkv, d)[:s] for c in (k_cache, v_cache))
        for h in range(H):
            first = [0, 3, 7][b]
            qs = np.concatenate([np.zeros((s - m, d)), q[first:first + m, h]])
            fo, top, total = oracle.forward_head(qs, k[:, h // 2], v[:, h // 2], 0.3, True, window)
            assert np.allclose(o[first:first + m, h], fo[s - m:], atol=1e-12)
            assert np.allclose(lse[first:first + m, h], (top + np.log(total))[s - m:], atol=1e-12)
    assert np.all(o[7:] == 0) and np.all(lse[7:] == -np.inf) and n.tolist()[:3] == ([7, 8, 9] if not window else [3] * 3)


def test_requests_shorter_than_their_rows():
    rng = np.random.default_rng(4)
    k_cache, v_cache = rng.normal(size=(2, 3, 2, 1, 8))
    q = rng.normal(size=(5, 1, 8))
    o, lse, _, _, n = paged.extend(q, k_cache, v_cache, [[0, 1], [2, -1]], [2, 1], [0, 4, 7], 1.0)
    assert n.tolist() == [0, 0, 1, 2, 0] and np.all(lse[[0, 1, 4]] == -np.inf) and np.all(np.isfinite(lse[2:4]))


def P(i):
    return ctypes.c_void_p(i << 40)


def _rc(lib, **kw):
    a = dict(q=P(1), qs=512, kc=P(2), vc=P(3), kind=0, k_scale=None, v_scale=None, page_stride=4096, slot_stride=256,
             head_stride=128, pages=8, page=16, table=P(4), table_stride=8, width=8, seq=P(5), cu=P(6), batch=2, n=4,
             heads=4, heads_kv=2, dim=128, window=0, scale=1.0, o=P(7), lse=P(8), ws=P(9), bytes=1 << 30)
    a.update(kw)
    return lib.fa_extend(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dim=96), 2, b"head_dim"), (dict(kind=2), 1, b"kv_type"), (dict(heads_kv=0), 1, b"heads_kv"),
    (dict(heads=3), 1, b"multiple"), (dict(heads=0), 1, b"multiple"), (dict(batch=-1), 1, b"batch"),
    (dict(n=-1), 1, b"num_tokens"), (dict(window=-1), 1, b"window"), (dict(scale=float("inf")), 1, b"scale"),
    (dict(width=-1), 1, b"max_pages"), (dict(width=1 << 30), 2, b"too long"), (dict(table_stride=-1), 1, b"table_stride"),
    (dict(qs=500), 1, b"q_row_stride"), (dict(qs=516), 1, b"q_row_stride"), (dict(q=None), 1, b"NULL"),
    (dict(o=None), 1, b"NULL"), (dict(cu=None), 1, b"NULL"), (dict(seq=None), 1, b"NULL"), (dict(table=None), 1, b"NULL"),
    (dict(kc=None), 1, b"NULL"), (dict(q=ctypes.c_void_p(8)), 1, b"aligned"), (dict(cu=ctypes.c_void_p(2)), 1, b"aligned"),
    (dict(lse=ctypes.c_void_p(2)), 1, b"aligned"), (dict(o=P(1)), 1, b"overlap"), (dict(ws=None), 1, b"workspace"),
    (dict(bytes=100), 1, b"workspace"), (dict(ws=ctypes.c_void_p(8)), 1, b"aligned"),
    (dict(n=1 << 30), 2, b"too many"), (dict(k_scale=P(1)), 1, b"e4m3"), (dict(slot_stride=64), 1, b"slot_stride")])
def test_refusals(lib, kw, code, word):
    assert _rc(lib, **kw) == code
    assert word in lib.fa_last_error()


def test_units_that_the_costs_have_no_room_for(lib):
    """From 2^25 units on (a request with tokens and a key/value head, at least one
    each) the call is refused; requests without tokens, a padded batch's, are no
    units."""
    many = dict(heads=32, heads_kv=32, qs=4096, batch=1 << 20)
    assert _rc(lib, **many, n=1 << 20) == 2 and b"too many" in lib.fa_last_error()
    assert _rc(lib, **{**many, "batch": 1 << 25, "heads": 1, "heads_kv": 1, "qs": 128}, n=1 << 25) == 2
    assert b"too many" in lib.fa_last_error()
    for batch in (1 << 28 | 1, (1 << 31) - 1):   # nor can so many be looked at
        assert _rc(lib, **{**many, "batch": batch}, n=100) == 2 and b"too many" in lib.fa_last_error()
    for batch in (1 << 20, 1 << 28):
        # passes, to the next refusal
        assert _rc(lib, **{**many, "batch": batch}, n=100, window=-1) == 1 and b"window" in lib.fa_last_error()


SHIFT = """
#include <cstdio>
#include "extend_shape.h"
int main() {
  long long units, keys;
  int bits;
  while (std::scanf("%lld %lld %d", &units, &keys, &bits) == 3) std::printf("%d\\n", fa::extend::cost_shift(units, keys, bits));
}
"""


def test_costs_of_any_call_fit(tmp_path):
    """The smallest step from a block's keys on with which the costs of all units
    that are not refused stay below 2^30."""
    (tmp_path / "main.cpp").write_text(SHIFT)
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_backward_sm_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I" + csrc, str(tmp_path / "main.cpp"), "-o",
                    str(tmp_path / "main")], check=True)
    units = [0, 1, 2, 1000, 1 << 20, (1 << 24) - 1, 1 << 24, (1 << 25) - 1]
    keys = [0, 1, 127, 128, 5000, 1 << 20, 0x7fff0000, 0x7fff0000 + 0x7ff00000]
    calls = [(u, k, b) for u in units for k in keys for b in (6, 7)]
    text = "".join("%d %d %d\n" % c for c in calls)
    out = subprocess.run([str(tmp_path / "main")], input=text, capture_output=True, text=True, check=True, timeout=20)
    shifts = [int(x) for x in out.stdout.split()]
    assert len(shifts) == len(calls)
    for (u, k, b), s in zip(calls, shifts):
        most = lambda shift: u * (3 * (k >> shift) + 32)  # noqa: E731
        assert most(s) < 1 << 30 and b <= s <= 63
        # one less would not do (the quotient is rounded down: as much as a unit's cost away)
        assert s == b or most(s - 1) + 3 * (k >> (s - 1)) + 32 >= 1 << 30


def test_nothing_succeeds(lib):
    assert _rc(lib, n=0, q=None, o=None, cu=None, seq=None, ws=None) == 0 and lib.fa_last_error() == b""


def test_workspace_size(lib):
    import attention_backward_sm_gb300 as fab
    for d in (64, 128, 256):
        assert fab.fa_extend_workspace_size(d) == lib.fa_extend_workspace_size(d) > 0
    with pytest.raises(fab.FabwdError) as e:
        fab.fa_extend_workspace_size(96)
    assert e.value.code == 2
