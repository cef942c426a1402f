"""Rotation by positions without a GPU: the oracle's pins, the frequencies, and
the refusals of the C entry points and of the binding (all before anything
touches the device)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import rope


@pytest.fixture(scope="module")
def lib():
    from attention_backward_sm_gb300 import build
    build.build()
    from attention_backward_sm_gb300 import _lib
    return _lib.load()


def fab():
    import attention_backward_sm_gb300 as m
    return m


# ------------------------------------------------------------------ oracle
def test_rotation_worked_by_hand():
    """A quarter turn per position: (1, 0) goes to (0, 1), (-1, 0), ..."""
    theta = np.array([math.pi / 2])
    x = np.zeros((4, 1, 6))
    x[..., 0], x[..., 5] = 1.0, 7.0
    for half in (True, False):   # one pair: values 0 and 1 in both layouts
        y = rope.rotate(x, np.arange(4), theta, half, 2.0)
        assert np.allclose(y[:, 0, :2], [[2, 0], [0, 2], [-2, 0], [0, -2]], atol=1e-12)
        assert np.all(y[..., 5] == 7) and np.all(y[..., 2:5] == 0)


@pytest.mark.parametrize("half", [True, False])
def test_scores_depend_on_distances_alone(half):
    rng = np.random.default_rng(0)
    theta = rope.frequencies(8)
    q, k = rng.normal(size=(2, 1, 1, 12))
    at = lambda p, x: rope.rotate(x, [p], theta, half)[0, 0]  # noqa: E731
    assert np.isclose(at(7, q) @ at(3, k), at(1004, q) @ at(1000, k), atol=1e-12)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_gradient_against_differences(half, weighted):
    rng = np.random.default_rng(1)
    T, H, d, eps = 3, 2, 10, 1e-3
    x, dy = rng.normal(size=(2, T, H, d))
    w = rng.normal(size=d) if weighted else None
    theta, pos, mscale = rope.frequencies(6), [0, 5, -3], 1.3
    loss = lambda x, w: (rope.forward(x, pos, theta, half, mscale, w, eps) * dy).sum()  # noqa: E731
    dx, dw = rope.backward(dy, x, pos, theta, half, mscale, w, eps)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert np.isclose((loss(x + e, w) - loss(x - e, w)) / (2 * h), dx[i], atol=1e-7)
    if weighted:
        for i in range(d):
            e = np.zeros(d)
            e[i] = h
            assert np.isclose((loss(x, w + e) - loss(x, w - e)) / (2 * h), dw[i], atol=1e-7)


# ------------------------------------------------------------------ frequencies
@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(factor=8.0),
                                dict(factor=4.0, original_len=4096),
                                dict(factor=8.0, original_len=8192, low=1.0, high=4.0)])
@pytest.mark.parametrize("rotary", [16, 64, 256])
def test_frequencies_in_turns(rotary, kw):
    """The 64-bit fraction is off by the rounding of its float64 value: 2^-53 of
    theta and of 2 pi and of their quotient, and half a unit of 2^-64."""
    got = fab().rope_freqs(rotary, device="cpu", **kw)
    want = rope.frequencies(rotary, **kw) / (2 * math.pi)
    turns = np.array([(int(v) % (1 << 64)) / 2.0 ** 64 for v in got])
    assert got.dtype == torch.int64 and got.shape == (rotary // 2,)
    assert np.all(np.abs(turns - want) <= 8 * 2.0 ** -53 * want + 2.0 ** -64)


def test_given_frequencies_wrap_at_a_turn():
    """More than a turn per position counts modulo 1, a negative one the other way."""
    f = fab().rope_freqs(4, inv_freq=[2 * math.pi * 1.25, -2 * math.pi * 0.25], device="cpu")
    assert [round((int(v) % (1 << 64)) / 2.0 ** 64, 12) for v in f] == [0.25, 0.75]
    assert fab().rope_freqs(0, device="cpu").numel() == 0


@pytest.mark.parametrize("kw", [dict(rotary_dim=15), dict(rotary_dim=-2), dict(rotary_dim=16, factor=0.0),
                                dict(rotary_dim=16, factor=float("nan")), dict(rotary_dim=16, base=0.0),
                                dict(rotary_dim=16, original_len=-1),
                                dict(rotary_dim=16, original_len=10, low=2.0, high=2.0),
                                dict(rotary_dim=16, inv_freq=[1.0]),
                                dict(rotary_dim=4, inv_freq=[1.0, float("inf")])])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        fab().rope_freqs(device="cpu", **kw)


# ------------------------------------------------------------------ C refusals
# Addresses that are never dereferenced: the checks fail first.
def P(i):
    return ctypes.c_void_p(i << 32)


def _rope_rc(lib, **kw):
    a = dict(q=P(1), k=P(2), qs=512, ks=256, pos=P(3), freqs=P(4), rotary=128, layout=0, mscale=1.0, qw=None, kw=None,
             wt=0, eps=1e-6, n=4, heads=4, heads_kv=2, dim=128, qo=P(5), ko=P(6), qos=512, kos=256)
    a.update(kw)
    return lib.fa_qk_rope(*a.values(), None)


COMMON = [
    (dict(dim=96), 2, b"head_dim"), (dict(rotary=24), 2, b"rotary_dim"), (dict(rotary=144), 2, b"rotary_dim"),
    (dict(rotary=-16), 2, b"rotary_dim"), (dict(layout=2), 1, b"layout"), (dict(wt=2), 1, b"weight_type"),
    (dict(mscale=float("inf")), 1, b"mscale"), (dict(eps=-1.0), 1, b"eps"), (dict(eps=float("nan")), 1, b"eps"),
    (dict(n=-1), 1, b"num_tokens"), (dict(heads=-1), 1, b"heads"), (dict(pos=None), 1, b"positions"),
    (dict(freqs=None), 1, b"freqs"), (dict(freqs=ctypes.c_void_p(4)), 1, b"aligned"),
    (dict(qw=ctypes.c_void_p(3)), 1, b"weight"), (dict(wt=1, kw=ctypes.c_void_p(2)), 1, b"weight"),
]


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(qs=504), 1, b"q_row_stride"), (dict(qs=516), 1, b"q_row_stride"), (dict(kos=128), 1, b"k_out_row_stride"),
    (dict(q=None), 1, b"q is NULL"), (dict(ko=None), 1, b"k_out is NULL"), (dict(q=ctypes.c_void_p(8)), 1, b"aligned"),
    (dict(qo=P(1), qos=520), 1, b"overlap"), (dict(qo=ctypes.c_void_p((1 << 32) + 16)), 1, b"overlap"),
    (dict(qo=P(2)), 1, b"overlap"), (dict(ko=P(1)), 1, b"overlap"), (dict(qo=P(6)), 1, b"overlap"),
    (dict(heads=1 << 20), 2, b"too large")])
def test_rope_refusals(lib, kw, code, word):
    assert _rope_rc(lib, **kw) == code
    assert word in lib.fa_last_error()


def test_rope_slices_of_one_buffer_do_not_overlap(lib):
    """Queries and keys of one projection, written in place of themselves and
    into columns of their own, pass the checks (an empty call is made of them)."""
    base = 1 << 32
    at = lambda e: ctypes.c_void_p(base + 2 * e)  # noqa: E731
    ok = dict(q=at(0), qs=2048, k=at(512), ks=2048, qo=at(0), qos=2048, ko=at(512), kos=2048)
    for n in (1, 4):
        # the checks of rows come before the device's
        assert _rope_rc(lib, n=n, **ok) in (0, 2, 3) and b"overlap" not in lib.fa_last_error()
        assert _rope_rc(lib, n=n, **{**ok, "qo": at(1024)}) in (0, 2, 3) and b"overlap" not in lib.fa_last_error()
        assert _rope_rc(lib, n=n, **{**ok, "qo": at(8)}) == 1 and b"overlap" in lib.fa_last_error()
        assert _rope_rc(lib, n=n, **{**ok, "ko": at(256)}) == 1 and b"overlap" in lib.fa_last_error()
    # a row that wraps into the next row's first columns
    assert _rope_rc(lib, n=4, **{**ok, "qo": at(2048 - 256)}) == 1 and b"overlap" in lib.fa_last_error()


def test_rope_of_nothing_succeeds(lib):
    none = dict(q=None, k=None, qo=None, ko=None, pos=None, freqs=None)
    assert _rope_rc(lib, n=0, **none) == 0 and lib.fa_last_error() == b""
    assert _rope_rc(lib, heads=0, heads_kv=0, **{**none, "pos": P(3), "freqs": P(4)}) == 0


def _bwd_rc(lib, **kw):
    a = dict(gq=P(1), gk=P(2), gqs=512, gks=256, q=P(7), k=P(8), qs=512, ks=256, pos=P(3), freqs=P(4), rotary=128,
             layout=0, mscale=1.0, qw=P(9), kw=P(10), wt=0, eps=1e-6, n=4, heads=4, heads_kv=2, dim=128, dq=P(5),
             dk=P(6), dqs=512, dks=256, dqw=P(11), dkw=P(12), ws=P(13), bytes=1 << 22)
    a.update(kw)
    return lib.fa_qk_rope_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(gqs=508), 1, b"dq_out_row_stride"), (dict(gk=None), 1, b"dk_out is NULL"), (dict(q=None), 1, b"q is NULL"),
    (dict(ks=128), 1, b"k_row_stride"), (dict(dq=None), 1, b"dq is NULL"), (dict(dk=ctypes.c_void_p(8)), 1, b"aligned"),
    (dict(dqw=None), 1, b"weight's gradient"), (dict(dkw=ctypes.c_void_p(2)), 1, b"aligned"),
    (dict(ws=None), 1, b"workspace"), (dict(bytes=16), 1, b"workspace"), (dict(ws=ctypes.c_void_p(8)), 1, b"aligned"),
    (dict(dq=P(7)), 1, b"overlap"), (dict(dk=P(5)), 1, b"overlap"), (dict(dq=P(1), dqs=520), 1, b"overlap")])
def test_rope_bwd_refusals(lib, kw, code, word):
    assert _bwd_rc(lib, **kw) == code
    assert word in lib.fa_last_error()


def test_rope_bwd_workspace(lib):
    for d in (64, 128, 256):
        assert fab().fa_qk_rope_bwd_workspace_size(d) == lib.fa_qk_rope_bwd_workspace_size(d) > 0
    with pytest.raises(fab().FabwdError) as e:
        fab().fa_qk_rope_bwd_workspace_size(80)
    assert e.value.code == 2


def _append_rc(lib, **kw):
    a = dict(q=P(1), k=P(2), v=P(14), qs=512, ks=256, vs=256, pos=P(3), freqs=P(4), rotary=128, layout=0, mscale=1.0,
             qw=None, kw=None, wt=0, eps=1e-6, n=4, heads=4, qo=P(5), qos=512, slots=P(15), kc=P(16), vc=P(17), kind=0,
             k_scale=None, v_scale=None, page_stride=4096, slot_stride=256, head_stride=128, pages=8, page=16,
             heads_kv=2, dim=128)
    a.update(kw)
    return lib.fa_qk_rope_append(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(kind=2), 1, b"kv_type"), (dict(heads_kv=0), 1, b"heads_kv"), (dict(pages=-1), 1, b"num_pages"),
    (dict(page=0), 1, b"page_size"), (dict(k_scale=P(1)), 1, b"e4m3"), (dict(slot_stride=260), 1, b"slot_stride"),
    (dict(vs=128), 1, b"v_row_stride"), (dict(v=None), 1, b"v is NULL"), (dict(slots=None), 1, b"NULL"),
    (dict(kc=None), 1, b"NULL"), (dict(slots=ctypes.c_void_p(4)), 1, b"aligned"), (dict(qo=P(14)), 1, b"overlap")])
def test_rope_append_refusals(lib, kw, code, word):
    assert _append_rc(lib, **kw) == code
    assert word in lib.fa_last_error()


# ------------------------------------------------------------------ binding refusals
def test_binding_refusals():
    f = fab()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    pos, fr = torch.zeros(3, dtype=torch.int32), f.rope_freqs(64, device="cpu")
    q, k = bf(3, 4, 64), bf(3, 2, 64)
    for args, kw, word in [
            ((q.float(), k, pos, fr), {}, "q must be bfloat16"), ((q, bf(2, 2, 64), pos, fr), {}, "k must be"),
            ((q, bf(3, 2, 128), pos, fr), {}, "k must be"), ((q[..., ::2], None, pos, fr), {}, "packed"),
            ((None, None, pos, fr), {}, "one at least"), ((q, k, pos.long(), fr), {}, "positions"),
            ((q, k, pos[:2], fr), {}, "positions"), ((q, k, pos, fr.int()), {}, "freqs"),
            ((q, k, pos, fr), dict(q_weight=torch.zeros(64, dtype=torch.float16)), "q_weight"),
            ((q, k, pos, fr), dict(q_weight=bf(32)), "q_weight"),
            ((q, k, pos, fr), dict(q_weight=bf(64), k_weight=torch.zeros(64)), "one type"),
            ((q, k, pos, fr), {}, "CUDA")]:
        with pytest.raises(ValueError, match=word):
            f.qk_rope(*args, **kw)
    with pytest.raises(ValueError, match="norm needs its input"):
        f.qk_rope_backward(q, k, pos, fr, q_weight=bf(64), k=k)
    with pytest.raises(ValueError, match="workspace"):
        f.qk_rope_backward(q, k, pos, fr, workspace=torch.zeros(4, 4)[:, 0])
    cache = bf(2, 4, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    for args, word in [((q, None, k, pos, fr, cache, cache, slots), "must be tensors"),
                       ((q, k, k, pos, fr, cache, cache, slots.int()), "slots"),
                       ((q, k, k, pos, fr, cache, cache[:1], slots), "one shape"),
                       ((q, q, k, pos, fr, cache, cache, slots), "k must be"),
                       ((q, k, k, pos, fr, cache, cache, slots), "CUDA")]:
        with pytest.raises(ValueError, match=word):
            f.qk_rope_append(*args)
