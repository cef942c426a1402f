"""Paged cache operators without a GPU: the oracle's pins, and the refusals
of the C entry points and of the binding (all before anything touches the
device)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle
from oracle import paged
from paged_paths import PATHS


@pytest.fixture(scope="module")
def lib():
    from attention_backward_sm_gb300 import build
    build.build()
    from attention_backward_sm_gb300 import _lib
    return _lib.load()


# ------------------------------------------------------------------ oracle
def test_plan_worked_by_hand():
    """Pages of 4: request 0 holds 5 tokens on pages 7, 2 and gets 4; request
    1 is empty and gets none; request 2 is empty and gets 2."""
    table = [[7, 2, -1], [-1, -1, -1], [-1, -1, -1]]
    t, slots, pos, cu, after, nxt = paged.plan(table, [5, 0, 0], [4, 0, 2], [9, 4, 6], 4, 8)
    assert slots.tolist() == [9, 10, 11, 36, 16, 17, -1, -1]
    assert pos.tolist() == [5, 6, 7, 8, 0, 1, 0, 0]
    assert cu.tolist() == [0, 4, 4, 6] and after.tolist() == [9, 0, 2] and nxt == 2
    assert t.tolist() == [[7, 2, 9], [-1, -1, -1], [4, -1, -1]]


def test_e4m3_matches_torch_on_every_border():
    """All 8-bit values, the midpoints between neighbours and their float32
    neighbours, against torch's conversion."""
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    v = v[torch.isfinite(v)].sort().values
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1)])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged.e4m3(x.double().numpy()), want)
    assert paged.e4m3([1e9, -1e9, np.inf]).tolist() == [448, -448, 448] and np.isnan(paged.e4m3(np.nan))


@pytest.mark.parametrize("window", [0, 5])
def test_decode_is_the_last_row_of_the_forward(window):
    """Over a permuted paged copy of packed K, V, single-token attention is
    the last query row of the causal forward."""
    rng = np.random.default_rng(3)
    H, Hkv, d, ps = 4, 2, 8, 4
    lens = [1, 4, 11]
    width = 3
    k_cache, v_cache = rng.normal(size=(2, 12, ps, Hkv, d))
    order = rng.permutation(12)
    table = order[:9].reshape(3, width)
    q = rng.normal(size=(3, H, d))
    o, lse, _, _ = paged.decode(q, k_cache, v_cache, table, lens, 0.3, window)
    for b, n in enumerate(lens):
        k = k_cache[table[b]].reshape(-1, Hkv, d)[:n]
        v = v_cache[table[b]].reshape(-1, Hkv, d)[:n]
        for h in range(H):
            qs = np.zeros((n, d))
            qs[-1] = q[b, h]
            fo, m, l = oracle.forward_head(qs, k[:, h // 2], v[:, h // 2], 0.3, True, window)
            assert np.allclose(o[b, h], fo[-1], atol=1e-12)
            assert np.isclose(lse[b, h], m[-1] + np.log(l[-1]), atol=1e-12)


def test_decode_rows_without_keys_and_bad_pages():
    rng = np.random.default_rng(4)
    k_cache, v_cache = rng.normal(size=(2, 3, 2, 1, 8))
    q = rng.normal(size=(3, 1, 8))
    o, lse, _, _ = paged.decode(q, k_cache, v_cache, [[0, 1], [-1, 3], [-1, 2]], [0, 4, 4], 1.0)
    assert np.all(o[:2] == 0) and np.all(lse[:2] == -np.inf)
    only = paged.decode(q[2:], k_cache, v_cache, [[2]], [2], 1.0)
    assert np.allclose(o[2], only[0][0]) and np.isclose(lse[2, 0], only[1][0, 0])


# ------------------------------------------------------------------ C refusals
P = ctypes.c_void_p(16)   # never dereferenced: the checks fail first


def _plan_rc(lib, **kw):
    a = dict(table=P, stride=8, width=8, seq=P, new=ctypes.c_void_p(32), free=P, num_free=4, start=None, page=16,
             batch=2, tokens=4, slots=P, pos=P, cu=P, out=ctypes.c_void_p(64), next=ctypes.c_void_p(96))
    a.update(kw)
    return lib.fa_kv_plan(a["table"], a["stride"], a["width"], a["seq"], a["new"], a["free"], a["num_free"],
                          a["start"], a["page"], a["batch"], a["tokens"], a["slots"], a["pos"], a["cu"], a["out"],
                          a["next"], None)


@pytest.mark.parametrize("kw,word", [
    (dict(page=0), b"page_size"), (dict(batch=-1), b"batch"), (dict(tokens=-1), b"num_tokens"),
    (dict(num_free=-1), b"num_free"), (dict(width=-1), b"max_pages"), (dict(stride=7), b"table_stride"),
    (dict(table=None), b"NULL"), (dict(seq=None), b"NULL"), (dict(free=None), b"NULL"), (dict(slots=None), b"NULL"),
    (dict(cu=None), b"NULL"), (dict(next=None), b"NULL"), (dict(out=P), b"seq_lens_out"),
    (dict(start=ctypes.c_void_p(96)), b"free_start"), (dict(slots=ctypes.c_void_p(20)), b"aligned"),
    (dict(pos=ctypes.c_void_p(18)), b"aligned")])
def test_plan_refusals(lib, kw, word):
    assert _plan_rc(lib, **kw) == 1
    assert word in lib.fa_last_error()


def _append_rc(lib, **kw):
    a = dict(k=P, v=P, ks=256, vs=256, slots=P, n=4, kc=P, vc=P, kind=0, k_scale=None, v_scale=None, page_stride=4096,
             slot_stride=256, head_stride=128, pages=8, page=16, heads_kv=2, dim=128)
    a.update(kw)
    return lib.fa_kv_append(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dim=96), 2, b"head_dim"), (dict(kind=2), 1, b"kv_type"), (dict(heads_kv=0), 1, b"heads_kv"),
    (dict(pages=-1), 1, b"num_pages"), (dict(page=0), 1, b"page_size"), (dict(k_scale=P), 1, b"e4m3"),
    (dict(page_stride=64), 1, b"page_stride"), (dict(slot_stride=260), 1, b"slot_stride"),
    (dict(head_stride=0), 1, b"head_stride"), (dict(kind=1, head_stride=136), 1, b"head_stride"),
    (dict(kc=ctypes.c_void_p(8)), 1, b"aligned"), (dict(n=-1), 1, b"num_tokens"), (dict(ks=128), 1, b"k_row_stride"),
    (dict(vs=260), 1, b"v_row_stride"), (dict(k=None), 1, b"NULL"), (dict(slots=None), 1, b"NULL"),
    (dict(v=ctypes.c_void_p(8)), 1, b"aligned"), (dict(slots=ctypes.c_void_p(4)), 1, b"aligned")])
def test_append_refusals(lib, kw, code, word):
    assert _append_rc(lib, **kw) == code
    assert word in lib.fa_last_error()


def test_append_of_nothing_succeeds(lib):
    assert _append_rc(lib, n=0, k=None, v=None, slots=None) == 0
    assert lib.fa_last_error() == b""


def _decode_rc(lib, **kw):
    a = dict(q=P, qs=512, kc=P, vc=P, kind=0, k_scale=None, v_scale=None, page_stride=4096, slot_stride=256,
             head_stride=128, pages=8, page=16, table=P, table_stride=4, width=4, seq=P, batch=2, heads=4, heads_kv=2,
             dim=128, window=0, scale=0.1, o=ctypes.c_void_p(1 << 20), lse=P, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return lib.fa_decode(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dim=32), 2, b"head_dim"), (dict(heads=3), 1, b"multiple"), (dict(heads=0), 1, b"multiple"),
    (dict(batch=-1), 1, b"batch"), (dict(window=-1), 1, b"window"), (dict(scale=float("nan")), 1, b"scale"),
    (dict(scale=float("inf")), 1, b"scale"), (dict(width=-1), 1, b"max_pages"),
    (dict(width=1 << 20, page=1 << 20), 2, b"too long"), (dict(table_stride=-4), 1, b"table_stride"),
    (dict(qs=256), 1, b"q_row_stride"), (dict(qs=516), 1, b"q_row_stride"), (dict(q=None), 1, b"NULL"),
    (dict(seq=None), 1, b"NULL"), (dict(table=None), 1, b"NULL"), (dict(kc=None), 1, b"NULL"),
    (dict(o=ctypes.c_void_p(8)), 1, b"aligned"), (dict(seq=ctypes.c_void_p(18)), 1, b"aligned"),
    (dict(o=P), 1, b"overlap"), (dict(o=ctypes.c_void_p(16 + 1024)), 1, b"overlap"),
    (dict(heads=1025, heads_kv=1, qs=1025 * 128), 2, b"1024"),
    (dict(batch=1 << 20, width=1 << 14), 2, b"too many"),
    (dict(heads=1 << 20, qs=1 << 27), 2, b"too large"),
    (dict(kind=0, v_scale=P), 1, b"e4m3"), (dict(slot_stride=100), 1, b"slot_stride")])
def test_decode_refusals(lib, kw, code, word):
    assert _decode_rc(lib, **kw) == code
    assert word in lib.fa_last_error()


def test_decode_workspace_size(lib):
    assert lib.fa_decode_workspace_size(4, 6, 4, 128) == 0 and b"multiple" in lib.fa_last_error()
    assert lib.fa_decode_workspace_size(4, 8, 4, 96) == 0 and b"head_dim" in lib.fa_last_error()
    n = lib.fa_decode_workspace_size(64, 32, 8, 128)
    assert lib.fa_last_error() == b""
    if n:   # too little of it, none of it and a misaligned one are refused
        kw = dict(batch=64, heads=32, heads_kv=8, page_stride=16384, slot_stride=1024, qs=4096)
        assert _decode_rc(lib, ws_bytes=n - 1, **kw) == 1 and b"workspace" in lib.fa_last_error()
        assert _decode_rc(lib, ws=None, **kw) == 1 and b"workspace" in lib.fa_last_error()
        assert _decode_rc(lib, ws=ctypes.c_void_p(8), **kw) == 1 and b"workspace" in lib.fa_last_error()


def test_decode_of_no_requests_succeeds(lib):
    assert _decode_rc(lib, batch=0, q=None, o=None, seq=None, table=None) == 0


# ------------------------------------------------------------------ binding refusals
def _tensors():
    return dict(q=torch.zeros(2, 4, 64, dtype=torch.bfloat16), k_cache=torch.zeros(6, 8, 2, 64, dtype=torch.bfloat16),
                v_cache=torch.zeros(6, 8, 2, 64, dtype=torch.bfloat16),
                block_table=torch.zeros(2, 3, dtype=torch.int32), seq_lens=torch.ones(2, dtype=torch.int32))


@pytest.mark.parametrize("change,word", [
    ({}, "CUDA"),
    (dict(q=torch.zeros(2, 4, 64)), "bfloat16"),
    (dict(q=torch.zeros(2, 4, 32, dtype=torch.bfloat16)), "head_dim"),
    (dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16)), "q must"),
    (dict(q=torch.zeros(2, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), "packed"),
    (dict(q=torch.zeros(2, 256, dtype=torch.bfloat16)), "q must"),
    (dict(v_cache=torch.zeros(6, 8, 1, 64, dtype=torch.bfloat16)), "one shape"),
    (dict(v_cache=torch.zeros(6, 8, 2, 64, dtype=torch.float16)), "float8"),
    (dict(v_cache=torch.zeros(6, 2, 8, 64, dtype=torch.bfloat16).transpose(1, 2)), "strides"),
    (dict(block_table=torch.zeros(2, 3, dtype=torch.int64)), "block_table"),
    (dict(block_table=torch.zeros(3, 2, dtype=torch.int32).t()), "contiguous rows"),
    (dict(seq_lens=torch.ones(3, dtype=torch.int32)), "seq_lens"),
    (dict(seq_lens=torch.ones(2)), "seq_lens"),
    (dict(k_scale=torch.ones(3)), "k_scale"),
    (dict(v_scale=torch.ones(2, dtype=torch.float64)), "v_scale")])
def test_decode_binding_refusals(lib, change, word):
    import attention_backward_sm_gb300 as fab
    with pytest.raises((ValueError, fab.FabwdError), match=word):
        fab.decode(**{**_tensors(), **change}, scale=0.1)


def test_append_and_plan_binding_refusals(lib):
    import attention_backward_sm_gb300 as fab
    t = _tensors()
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        fab.kv_append(k, k, t["k_cache"], t["v_cache"], slots)
    with pytest.raises(ValueError, match="slots"):
        fab.kv_append(k, k, t["k_cache"], t["v_cache"], slots.int())
    with pytest.raises(ValueError, match="k must"):
        fab.kv_append(k[:4], k, t["k_cache"], t["v_cache"], slots)
    i32 = dict(dtype=torch.int32)
    args = [t["block_table"], t["seq_lens"], torch.ones(2, **i32), torch.zeros(4, **i32)]
    with pytest.raises(ValueError, match="CUDA"):
        fab.kv_plan(*args, 8, 2)
    with pytest.raises(ValueError, match="new_lens"):
        fab.kv_plan(*args[:2], torch.ones(3, **i32), args[3], 8, 2)
    with pytest.raises(ValueError, match="free_start"):
        fab.kv_plan(*args, 8, 2, free_start=torch.zeros(2, **i32))


@pytest.mark.parametrize("args,code", [((4, 8, 4, 96), 2), ((4, 6, 4, 128), 1), ((-1, 8, 4, 128), 1), ((4, 0, 1, 96), 1)])
def test_workspace_size_binding_raises_the_code_of_fa_decode(lib, args, code):
    import attention_backward_sm_gb300 as fab
    with pytest.raises(fab.FabwdError) as e:
        fab.fa_decode_workspace_size(*args)
    assert e.value.code == code
    batch, heads, heads_kv, dim = args
    assert _decode_rc(lib, batch=batch, heads=heads, heads_kv=heads_kv, dim=dim) == (2 if dim == 96 else code)


# ------------------------------------------------------------------ what a call launches
SHAPES = r"""
#include <cstdio>
#include "decode_shape.h"
using namespace fa::decode;

template <int D, bool E>
void show(const Call& c) {
  Launch lc = split_heads(c.heads, c.heads_kv, c.head_dim, c.e4m3);
  with_shape<D, E>(c, lc, [&](auto nh, auto hw) {
    using Sh = Shape<D, E, decltype(nh)::value, decltype(hw)::value>;
    set_blocks<Sh, decltype(hw)::value>(c, lc);
    // what the launch writes: cuts, and two partial results per block
    const size_t used = static_cast<size_t>(lc.blocks) * lc.chunks *
                        (sizeof(Cut) + 2 * part_floats(lc.group * lc.rows, D) * sizeof(float));
    std::printf("%d %d %d %d %d %d %d %d %d %zu %zu\n", decltype(nh)::value, decltype(hw)::value, lc.rows, lc.chunks,
                lc.blocks, 1 << lc.tile_shift, lc.by_unit, lc.joined, Sh::kTile, used,
                workspace_bytes(c.batch, c.heads, c.heads_kv, c.head_dim));
    return 0;
  });
}

int main() {
  Call c;
  int e4m3;
  while (std::scanf("%d %d %d %d %d %d %d %d", &c.batch, &c.heads, &c.heads_kv, &c.head_dim, &e4m3, &c.keys, &c.window,
                    &c.sms) == 8) {
    c.e4m3 = e4m3 != 0;
    if (c.head_dim == 64) c.e4m3 ? show<64, true>(c) : show<64, false>(c);
    if (c.head_dim == 128) c.e4m3 ? show<128, true>(c) : show<128, false>(c);
    if (c.head_dim == 256) c.e4m3 ? show<256, true>(c) : show<256, false>(c);
  }
}
"""


class Shape:
    def __init__(self, line):
        (self.nh, self.hw, self.rows, self.chunks, self.blocks, self.tile, self.by_unit, self.joined, self.kernel_tile,
         self.used, self.workspace) = map(int, line.split())


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """shapes(calls): what each of (batch, heads, heads_kv, head_dim, e4m3,
    keys, window, SMs) launches, from the library's own header."""
    at = tmp_path_factory.mktemp("shapes")
    (at / "main.cpp").write_text(SHAPES)
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_backward_sm_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I" + csrc, str(at / "main.cpp"), "-o", str(at / "main")],
                   check=True)

    def ask(calls):
        text = "".join(" ".join(map(str, c)) + "\n" for c in calls)
        out = subprocess.run([str(at / "main")], input=text, capture_output=True, text=True, check=True).stdout
        return [Shape(line) for line in out.splitlines()]
    return ask


@pytest.mark.parametrize("path", PATHS, ids=str)
def test_decode_takes_the_path_that_its_case_is_there_for(shapes, path):
    assert max(path.lens) <= path.width * path.page
    s, = shapes([(path.batch, path.heads, path.heads_kv, path.dim, int(path.kv == "e4m3"), path.width * path.page, 0, 152)])
    tiles = sum(max(1, -(-n // s.tile)) for n in path.lens) * (path.heads_kv // s.hw)
    assert (s.nh, s.hw, s.chunks) == (path.nh, path.hw, path.chunks)
    assert ("none" if not s.joined else "unit" if s.by_unit else "cut") == path.join
    assert (tiles >= 4 * s.blocks) == path.cost
    assert s.tile == s.kernel_tile


def test_decode_workspace_holds_what_any_launch_writes(lib, shapes):
    """For every shape of heads, either cache, tables and windows of one key to
    a million, few and many requests, fewer and more SMs than a GB300's: cuts
    and partial results of all blocks fit, and the size is the C entry's."""
    calls = []
    for dim in (64, 128, 256):
        for heads_kv in (1, 2, 3, 4, 6, 8, 16, 40):
            for group in [*range(1, 35), 47, 48, 49, 63, 64, 65, 127, 128, 255, 300, 512, 1000, 1024]:
                for e4m3 in (0, 1):
                    for batch, keys, window, sms in ((1, 1, 0, 152), (1, 1 << 20, 0, 152), (3, 4096, 0, 148),
                                                     (64, 8192, 0, 152), (64, 131072, 100, 152), (300, 64, 0, 152),
                                                     (4000, 131072, 0, 152), (64, 8192, 0, 160), (64, 1 << 18, 0, 2),
                                                     (700, 30, 0, 152), (700, 17, 0, 400)):
                        calls.append((batch, heads_kv * group, heads_kv, dim, e4m3, keys, window, sms))
    for c, s in zip(calls, shapes(calls)):
        assert s.used <= s.workspace == lib.fa_decode_workspace_size(c[0], c[1], c[2], c[3]), c
        assert s.blocks >= 1 and s.rows * s.chunks >= c[1] // c[2] > s.rows * (s.chunks - 1), c
        assert s.tile == s.kernel_tile


@pytest.mark.parametrize("heads,heads_kv,dim", [(64, 4, 256), (32, 8, 128), (16, 16, 64), (8, 1, 256), (300, 1, 128)])
def test_decode_workspace_is_what_some_launch_needs(shapes, lib, heads, heads_kv, dim):
    """No shape's blocks and heads per tile are multiplied with another's."""
    calls = [(batch, heads, heads_kv, dim, e4m3, keys, 0, 152) for e4m3 in (0, 1)
             for batch, keys in ((1, 1 << 20), (1, 4096), (64, 1 << 17), (700, 30))]
    assert lib.fa_decode_workspace_size(1, heads, heads_kv, dim) <= max(s.used for s in shapes(calls)) + 255


# ------------------------------------------------------------------ more refusals
@pytest.mark.parametrize("call,kw,code,word", [
    ("plan", dict(out=ctypes.c_void_p(32)), 1, b"seq_lens_out"), ("plan", dict(new=None), 1, b"NULL"),
    ("plan", dict(out=None), 1, b"NULL"), ("plan", dict(pos=None), 1, b"NULL"),
    ("plan", dict(table=ctypes.c_void_p(18)), 1, b"aligned"), ("plan", dict(next=ctypes.c_void_p(98)), 1, b"aligned"),
    ("append", dict(heads_kv=40000, ks=40000 * 128, vs=40000 * 128), 2, b"too large"),
    ("append", dict(kind=1, k_scale=ctypes.c_void_p(18)), 1, b"aligned"),
    ("append", dict(kind=1, v_scale=ctypes.c_void_p(18)), 1, b"aligned"),
    ("append", dict(v_scale=P), 1, b"e4m3"), ("append", dict(vc=ctypes.c_void_p(24)), 1, b"aligned"),
    ("append", dict(v=None), 1, b"NULL"), ("append", dict(vc=None), 1, b"NULL"),
    ("decode", dict(lse=ctypes.c_void_p(18)), 1, b"aligned"), ("decode", dict(table=ctypes.c_void_p(18)), 1, b"aligned"),
    ("decode", dict(q=ctypes.c_void_p(24)), 1, b"aligned"), ("decode", dict(o=None), 1, b"NULL"),
    ("decode", dict(vc=None), 1, b"NULL"), ("decode", dict(kind=1, k_scale=ctypes.c_void_p(18)), 1, b"aligned"),
    ("decode", dict(kind=-1), 1, b"kv_type"), ("decode", dict(pages=-1), 1, b"num_pages"),
    ("decode", dict(page=0), 1, b"page_size"), ("decode", dict(heads_kv=0), 1, b"heads_kv")])
def test_refusals_of_the_other_arguments(lib, call, kw, code, word):
    assert {"plan": _plan_rc, "append": _append_rc, "decode": _decode_rc}[call](lib, **kw) == code
    assert word in lib.fa_last_error()


def test_decode_refuses_a_workspace_that_is_too_small(lib):
    n = lib.fa_decode_workspace_size(64, 32, 8, 128)
    assert n >= 2 * 152 * (16 + 2 * 4 * 4 * 130)   # two partial results of a head group for a block on every SM, at least
    kw = dict(batch=64, heads=32, heads_kv=8, page_stride=16384, slot_stride=1024, qs=4096)
    for bad in (dict(ws_bytes=n - 1), dict(ws_bytes=0), dict(ws=None), dict(ws=ctypes.c_void_p(8))):
        assert _decode_rc(lib, **kw, **bad) == 1 and b"workspace" in lib.fa_last_error()


def test_binding_refuses_what_is_no_tensor_or_number(lib):
    import attention_backward_sm_gb300 as fab
    t = _tensors()
    with pytest.raises(ValueError, match="q must be a tensor"):
        fab.decode(**{**t, "q": [1.0]}, scale=0.1)
    with pytest.raises(TypeError):
        fab.decode(**t, scale="large")
    with pytest.raises(TypeError):
        fab.decode(**t, scale=0.1, window=1.5)
    with pytest.raises(ValueError, match="window does not fit"):
        fab.decode(**t, scale=0.1, window=1 << 40)
    i32 = dict(dtype=torch.int32)
    args = [t["block_table"], t["seq_lens"], torch.ones(2, **i32), torch.zeros(4, **i32)]
    with pytest.raises(ValueError, match="num_tokens"):
        fab.kv_plan(*args, 8, -1)
    with pytest.raises(ValueError, match="page_size does not fit"):
        fab.kv_plan(*args, 1 << 40, 2)
