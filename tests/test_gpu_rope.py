"""Rotation by positions on the GPU against the fp64 oracle.

Bounds per element (derived, not tuned).  u = 2^-8 is half a step of bf16 in
relation to the value.  In fp32:
  * an angle is off by 2^-24 of half a turn at most in its conversion and 2^-32
    turns before it, its sine and cosine by 2 ulp: together below 2^-21.5 each;
  * the norm's factor: the sum of d squares in a tree of 16 + log2(d / 16)
    additions (half of their 2^-24 each goes through the root), the division by
    d, eps, a root of 2 ulp, two products: below 2^-19 of the value;
so with S = mscale (|n_a| + |n_b|) of a value's pair
    |y - ref| <= u |ref| + 2^-18 S.
The gradient's parts take the same roundings twice and a mean over d more:
    |dx - ref| <= u |ref| + 2^-17 (S w + |u| mean(S w |u|)) / r,
and a weight's gradient sums N rows, N / 16 of them at most after one another
in one thread, the threads, warps and blocks in some 64 more additions:
    |dw - ref| <= (2^-17 + (N / 16 + 64) 2^-24) sum S |u|.
To an e4m3 cache half a step is 2^-4 of the value (2^-10 below 2^-6)."""
import threading

import numpy as np
import pytest
import torch

from oracle import paged, rope

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def fab():
    import attention_backward_sm_gb300 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


class Problem:
    def __init__(self, T, H, Hkv, d, rotary, half=True, norm="", weight=torch.bfloat16, mscale=1.0, seed=0, far=4096,
                 strided=True, eps=1e-6, freqs=None):
        g = torch.Generator().manual_seed(seed)
        bf = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
        fused = bf(T, H + 2 * Hkv, d)
        self.q, self.k, self.v = fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]
        if not strided:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.dq, self.dk = bf(T, H, d), bf(T, Hkv, d)
        self.pos = torch.randint(-far // 8, far, (T,), generator=g, dtype=torch.int32)
        self.w = {n: (1 + 0.3 * torch.randn(d, generator=g)).to(weight) if n in norm else None for n in "qk"}
        self.half, self.mscale, self.eps, self.rotary = half, mscale, eps, rotary
        self.freq_kw = freqs or {}
        self.theta = rope.frequencies(rotary, **self.freq_kw)

    def on(self):
        """The tensors on the device, slices of one buffer again."""
        H, Hkv = self.q.shape[1], self.k.shape[1]
        if self.q.is_contiguous() and self.q.shape[0] > 1:
            return self.q.to(DEV), self.k.to(DEV), self.v.to(DEV)
        fused = torch.cat([self.q, self.k, self.v], 1).to(DEV)
        return fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]

    def args(self):
        freqs = fab().rope_freqs(self.rotary, device=DEV, **self.freq_kw)
        kw = dict(layout=fab().FA_ROPE_HALF if self.half else fab().FA_ROPE_INTERLEAVED, mscale=self.mscale,
                  eps=self.eps, **{n + "_weight": None if w is None else w.to(DEV) for n, w in self.w.items()})
        return self.pos.to(DEV), freqs, kw

    def forward(self):
        q, k, _ = self.on()
        pos, freqs, kw = self.args()
        return fab().qk_rope(q, k, pos, freqs, **kw)

    def want(self, n):
        x, w = f64(getattr(self, n)), self.w[n]
        w = None if w is None else f64(w)
        ref = rope.forward(x, self.pos.numpy(), self.theta, self.half, self.mscale, w, self.eps)
        plain = x if w is None else rope.norm(x, w, self.eps)
        return ref, rope.spread(plain, self.theta, self.half, self.mscale)

    def check(self, got, n):
        ref, s = self.want(n)
        err = np.abs(f64(got) - ref)
        assert got.dtype == torch.bfloat16 and got.shape == getattr(self, n).shape
        assert np.all(err <= U * np.abs(ref) + 2.0 ** -18 * s), f"{n} off by {err.max():.3e}"

    def check_grad(self, got, got_w, n):
        dy, x, w = f64(getattr(self, "d" + n)), f64(getattr(self, n)), self.w[n]
        w = None if w is None else f64(w)
        ref, ref_w = rope.backward(dy, x, self.pos.numpy(), self.theta, self.half, self.mscale, w, self.eps)
        s = rope.spread(dy, self.theta, self.half, self.mscale)
        if w is None:
            assert got_w is None
            tol = 2.0 ** -18 * s
        else:
            r = np.sqrt((x * x).mean(-1, keepdims=True) + self.eps)
            u = np.abs(x) / r
            sw = s * np.abs(w)
            tol = 2.0 ** -17 * (sw + u * (sw * u).mean(-1, keepdims=True)) / r
            rows = x.shape[0] * x.shape[1]
            tol_w = (2.0 ** -17 + (rows / 16 + 64) * 2.0 ** -24) * (s * u).sum((0, 1))
            err = np.abs(f64(got_w) - ref_w)
            assert got_w.dtype == torch.float32
            assert np.all(err <= tol_w), f"d{n}_weight off by {err.max():.3e}"
        err = np.abs(f64(got) - ref)
        assert np.all(err <= U * np.abs(ref) + tol), f"d{n} off by {err.max():.3e}"

    def backward(self, **over):
        q, k, _ = self.on()
        pos, freqs, kw = self.args()
        return fab().qk_rope_backward(self.dq.to(DEV), self.dk.to(DEV), pos, freqs, q=q, k=k, **{**kw, **over})


SHAPES = [
    # T, H, Hkv, d, rotary
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (2, 8, 1, 256, 256), (3, 5, 1, 64, 16), (63, 7, 7, 128, 96),
    (64, 16, 4, 128, 128), (65, 3, 2, 256, 48), (777, 6, 2, 128, 64), (1217, 4, 4, 64, 48), (5001, 2, 1, 256, 240),
    (4865, 8, 2, 64, 64), (100, 12, 3, 128, 0)]


@pytest.mark.parametrize("half", [True, False], ids=["half", "interleaved"])
@pytest.mark.parametrize("norm", ["", "qk", "q", "k"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradient(shape, norm, half):
    p = Problem(*shape, half=half, norm=norm, mscale=1.0 if norm else 1.25, seed=sum(shape),
                weight=torch.float32 if shape[0] % 2 else torch.bfloat16, strided=shape[0] % 3 != 0)
    q, k = p.forward()
    p.check(q, "q")
    p.check(k, "k")
    dq, dk, dqw, dkw = p.backward()
    p.check_grad(dq, dqw, "q")
    p.check_grad(dk, dkw, "k")


@pytest.mark.parametrize("kw", [dict(factor=8.0), dict(factor=4.0, original_len=4096), dict(base=1e6)])
def test_far_positions_and_scaled_frequencies(kw):
    """Angles of positions up to 2^31 - 1: the oracle's 64-bit product of
    position and frequency is itself off by 2^31 2^-52 radians, far below the
    bound."""
    p = Problem(257, 4, 2, 128, 128, freqs=kw, mscale=1.1, seed=3)
    p.pos[:6] = torch.tensor([2 ** 31 - 1, -2 ** 31, 10 ** 9, 131071, 0, -1], dtype=torch.int32)
    for got, n in zip(p.forward(), "qk"):
        p.check(got, n)


@pytest.mark.parametrize("half", [True, False], ids=["half", "interleaved"])
def test_angles_are_finer_than_32_bits(half):
    """The weights' gradient of one row shows sines and cosines in fp32: with x = 1
    and dy = 1 in the first value of every pair they are cos t and -sin t.  Where
    they are small, an angle rounded to 24 bits (9e-8 radians) would stand out:
    off by 2^-20 of the value (the norm's factor and five roundings) and by 2^-32
    turns, of which 2^-28 radians leaves twice the room."""
    d = 256
    freqs, w = fab().rope_freqs(d), torch.ones(d, device=DEV)
    x = torch.ones(1, 1, d, dtype=torch.bfloat16, device=DEV)
    first = torch.arange(d) < d // 2 if half else torch.arange(d) % 2 == 0
    dy = first.bfloat16().to(DEV).view(1, 1, d)
    layout = fab().FA_ROPE_HALF if half else fab().FA_ROPE_INTERLEAVED
    seen = 0
    for position in (1, 7, 100, -1000, 4095, 50021, 65535):
        pos = torch.tensor([position], dtype=torch.int32, device=DEV)
        got = f64(fab().qk_rope_backward(dy, None, pos, freqs, layout=layout, q=x, q_weight=w)[2])
        t = position * rope.frequencies(d)
        ref = np.empty(d)
        ref[first.numpy()], ref[~first.numpy()] = np.cos(t), -np.sin(t)
        ref /= np.sqrt(1 + 1e-6)
        small = np.abs(ref) < 2.0 ** -5
        seen += small.sum()
        err = np.abs(got - ref)
        assert np.all(err[small] <= 2.0 ** -20 * np.abs(ref[small]) + 2.0 ** -28), f"off by {err[small].max():.3e}"
        assert np.all(err <= 2.0 ** -20)
    assert seen > 150


def test_one_tensor_alone():
    p = Problem(70, 4, 2, 128, 128, norm="qk", seed=4)
    q, k, _ = p.on()
    pos, freqs, kw = p.args()
    oq, none = fab().qk_rope(q, None, pos, freqs, **kw)
    assert none is None
    p.check(oq, "q")
    none, ok = fab().qk_rope(None, k, pos, freqs, **kw)
    assert none is None
    p.check(ok, "k")
    kw["q_weight"] = None
    none, dk, none2, dkw = fab().qk_rope_backward(None, p.dk.to(DEV), pos, freqs, k=k, **kw)
    assert none is None and none2 is None
    p.check_grad(dk, dkw, "k")


def test_nothing():
    pos, freqs = torch.zeros(0, dtype=torch.int32, device=DEV), fab().rope_freqs(64)
    e = torch.zeros(0, 3, 64, dtype=torch.bfloat16, device=DEV)
    q, k = fab().qk_rope(e, e, pos, freqs)
    assert q.shape == k.shape == e.shape
    w = torch.ones(64, device=DEV)
    dq, dk, dqw, dkw = fab().qk_rope_backward(e, e, pos, freqs, q=e, k=e, q_weight=w, k_weight=w)
    assert dq.shape == e.shape and torch.all(dqw == 0) and torch.all(dkw == 0)


@pytest.mark.parametrize("half", [True, False])
def test_in_place_and_strided_outputs(half):
    p = Problem(333, 6, 2, 128, 96, half=half, norm="qk", seed=5)
    want = p.forward()
    pos, freqs, kw = p.args()
    q, k, v = p.on()
    keep = v.clone()
    fab().fa_qk_rope(q, k, pos, freqs, q, k, **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep)
    q, k, _ = p.on()
    wide = torch.full((333, 20, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    got = fab().qk_rope(q, k, pos, freqs, out=(wide[:, 2:8], wide[:, 9:11]), **kw)
    assert got[0].data_ptr() == wide[:, 2:8].data_ptr()
    assert torch.equal(wide[:, 2:8], want[0]) and torch.equal(wide[:, 9:11], want[1])
    assert torch.all(wide[:, [0, 1, 8]] == 3) and torch.all(wide[:, 11:] == 3)
    # the gradient over its own input
    ref = p.backward()
    gq, gk = p.dq.to(DEV), p.dk.to(DEV)
    q, k, _ = p.on()
    w = torch.full((2, 128), 9.0, device=DEV)
    fab().fa_qk_rope_bwd(gq, gk, pos, freqs, gq, gk, w[0], w[1], q=q, k=k, **kw)
    for a, b in zip((gq, gk, w[0], w[1]), ref):
        assert torch.equal(a, b)


def test_values_that_are_not_numbers_stay_in_their_head():
    p = Problem(40, 3, 2, 64, 32, norm="qk", seed=6)
    clean = p.forward()
    p.q[7, 1, 5], p.k[9, 0, 60] = float("nan"), float("inf")
    q, k = p.forward()
    assert q[7, 1].isnan().all() and k[9, 0].isnan().any()
    q[7, 1], k[9, 0] = clean[0][7, 1], clean[1][9, 0]
    assert torch.equal(q, clean[0]) and torch.equal(k, clean[1])
    # without a norm only their pair is touched
    p = Problem(40, 3, 2, 64, 32, seed=6)
    clean = p.forward()[0]
    p.q[7, 1, 5] = float("nan")
    q = p.forward()[0]
    assert q[7, 1, [5, 21]].isnan().all()
    q[7, 1, [5, 21]] = clean[7, 1, [5, 21]]
    assert torch.equal(q, clean)


def test_rows_of_zeros():
    p = Problem(5, 2, 2, 64, 64, norm="qk", seed=7, eps=1e-5)
    p.q[2] = 0
    q, k = p.forward()
    assert torch.all(q[2] == 0)
    dq, dk, dqw, dkw = p.backward()
    p.check_grad(dq, dqw, "q")


def test_offsets_past_32_bits():
    """Rows so far apart that the last ones lie past 2^31 elements."""
    p = Problem(33, 4, 2, 128, 128, norm="qk", seed=8, strided=False)
    want, ref = p.forward(), p.backward()
    pos, freqs, kw = p.args()
    stride = 1 << 27
    big = torch.empty(33 * stride, dtype=torch.bfloat16, device=DEV)
    at = lambda o, h: big.as_strided((33, h, 128), (stride, 128, 1), o)  # noqa: E731
    q, k, qo, ko, gq, gk = (at(i * 4096, h) for i, h in enumerate((4, 2, 4, 2, 4, 2)))
    q.copy_(p.q)
    k.copy_(p.k)
    gq.copy_(p.dq)
    gk.copy_(p.dk)
    fab().qk_rope(q, k, pos, freqs, out=(qo, ko), **kw)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    got = fab().qk_rope_backward(gq, gk, pos, freqs, q=q, k=k, out=(qo, ko, ref[2].clone(), ref[3].clone()), **kw)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_weights_without_tokens_need_no_positions(dim):
    """The C entry with weights and no tokens: zeros as the weights' gradients;
    everything that belongs to tokens may be NULL."""
    from attention_backward_sm_gb300._lib import load
    f32, at = fab().FA_WEIGHT_F32, lambda t: t.data_ptr()  # noqa: E731
    w = torch.ones(2, dim, device=DEV)
    dw = torch.full((2, dim), 9.0, device=DEV)
    size = fab().fa_qk_rope_bwd_workspace_size(dim)
    work = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    rc = load().fa_qk_rope_bwd(None, None, 0, 0, None, None, 0, 0, None, None, dim, 0, 1.0, at(w[0]), at(w[1]), f32, 1e-6,
                               0, 4, 2, dim, None, None, 0, 0, at(dw[0]), at(dw[1]), at(work), size,
                               torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.all(dw == 0)


# ------------------------------------------------------------------ into the cache
def cache_of(pages, page, Hkv, d, kv, layout="plain"):
    t = torch.full((pages, page, Hkv, d), -2.0, device=DEV).to(torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn)
    if layout == "heads_first":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    return t


@pytest.mark.parametrize("layout", ["plain", "heads_first"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("norm", ["", "qk"])
@pytest.mark.parametrize("shape", [(1, 4, 1, 64, 64), (64, 32, 8, 128, 128), (77, 3, 3, 256, 64), (2500, 8, 2, 64, 32),
                                   (1300, 6, 6, 128, 112),
                                   # enough for the stream: whole and part chunks, more than 32 tokens to a warp
                                   (6500, 8, 4, 128, 128), (5001, 5, 3, 256, 128), (7001, 36, 9, 64, 64),
                                   (90001, 2, 1, 64, 32)], ids=str)
def test_append_is_rotation_then_append(shape, norm, kv, layout):
    T, H, Hkv, d, rotary = shape
    p = Problem(*shape, half=T % 2 == 0, norm=norm, seed=T)
    page, pages = 7, T // 7 + 5
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:T]
    if T > 4:
        slots[3], slots[T - 1] = -1, pages * page + 3   # outside the cache
    slots = slots.to(DEV)
    scales = {} if kv == "bf16" else {n: 0.01 + 0.01 * torch.rand(Hkv, device=DEV) for n in ("k_scale", "v_scale")}
    kc, vc, kc2, vc2 = (cache_of(pages, page, Hkv, d, kv, layout) for _ in range(4))
    q, k, v = p.on()
    pos, freqs, kw = p.args()
    qo = fab().qk_rope_append(q, k, v, pos, freqs, kc, vc, slots, **scales, **kw)
    want_q, want_k = fab().qk_rope(q, k, pos, freqs, **kw)
    fab().kv_append(want_k, v, kc2, vc2, slots, **scales)
    assert torch.equal(qo, want_q)
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(bits(vc), bits(vc2))
    ok = ((slots >= 0) & (slots < pages * page)).cpu()
    if kv == "bf16":
        assert torch.equal(bits(kc), bits(kc2))
        return
    # rounded once, from fp32: within half a step of the 64-bit value and its fp32 error
    ref, s = p.want("k")
    scale = f64(scales["k_scale"])[:, None]
    ref, s = ref / scale, s / scale
    held = f64(kc.reshape(-1, Hkv, d).float())[slots.cpu()[ok].numpy()]
    ref, s = ref[ok.numpy()], s[ok.numpy()]
    step = np.maximum(np.abs(ref) * 2.0 ** -4, 2.0 ** -10)
    near = np.abs(held - np.clip(ref, -448, 448)) <= step + 2.0 ** -18 * s
    assert near.all()
    # all but those next to the border of two values are the nearest one
    assert np.mean(held == paged.e4m3(ref)) > 0.999
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots.cpu()[ok]] = False
    assert torch.all(kc.reshape(-1, Hkv, d)[rest.to(DEV)].float() == -2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("weight", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("norm", ["q", "k"])
@pytest.mark.parametrize("T,H,Hkv,d,rotary", [(64, 8, 2, 128, 128), (5000, 12, 4, 128, 96), (6001, 4, 4, 256, 256),
                                              (9000, 16, 2, 64, 64)])
def test_append_with_one_norm(T, H, Hkv, d, rotary, norm, weight, kv):
    """A norm of one tensor only, either type of weights, outputs scaled: few rows
    and enough for the stream, which keep these in different places."""
    p = Problem(T, H, Hkv, d, rotary, half=T % 2 == 0, norm=norm, weight=weight, mscale=1.25, seed=T + d)
    page, pages = 16, T // 16 + 1
    slots = torch.arange(T, device=DEV)
    scales = {} if kv == "bf16" else {n: 0.01 + 0.01 * torch.rand(Hkv, device=DEV) for n in ("k_scale", "v_scale")}
    kc, vc = (cache_of(pages, page, Hkv, d, kv) for _ in range(2))
    q, k, v = p.on()
    pos, freqs, kw = p.args()
    p.check(fab().qk_rope_append(q, k, v, pos, freqs, kc, vc, slots, **scales, **kw), "q")
    held = kc.reshape(-1, Hkv, d)[:T]
    if kv == "bf16":
        p.check(held, "k")
        return
    ref, s = p.want("k")
    scale = f64(scales["k_scale"])[:, None]
    ref, s = ref / scale, s / scale
    err = np.abs(f64(held.float()) - np.clip(ref, -448, 448))
    assert np.all(err <= np.maximum(np.abs(ref) * 2.0 ** -4, 2.0 ** -10) + 2.0 ** -18 * s)


def test_append_in_place_and_without_pages():
    p = Problem(9, 2, 2, 64, 64, seed=9)
    pos, freqs, kw = p.args()
    q, k, v = p.on()
    want = fab().qk_rope(q, k, pos, freqs, **kw)[0]
    empty = torch.zeros(0, 4, 2, 64, dtype=torch.bfloat16, device=DEV)
    slots = torch.zeros(9, dtype=torch.int64, device=DEV)
    got = fab().qk_rope_append(q, k, v, pos, freqs, empty, empty, slots, out=q, **kw)
    assert got.data_ptr() == q.data_ptr() and torch.equal(q, want)


# ------------------------------------------------------------------ streams, graphs, threads
def test_captured_and_replayed():
    p = Problem(300, 8, 2, 128, 128, norm="qk", seed=10)
    pos, freqs, kw = p.args()
    q, k, _ = p.on()
    gq, gk = p.dq.to(DEV), p.dk.to(DEV)
    want, ref = p.forward(), p.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fab().qk_rope(q, k, pos, freqs, **kw)
        grads = fab().qk_rope_backward(gq, gk, pos, freqs, q=q, k=k, **kw)
    for _ in range(3):
        for t in (*out, *grads):
            t.fill_(7)
        graph.replay()
        for a, b in zip((*out, *grads), (*want, *ref)):
            assert torch.equal(a, b)
    # other positions in the same buffer
    p.pos += 17
    pos.copy_(p.pos)
    graph.replay()
    p.check(out[0], "q")
    p.check_grad(grads[1], grads[3], "k")


def test_another_stream():
    p = Problem(1000, 8, 2, 128, 128, norm="qk", seed=11)
    pos, freqs, kw = p.args()
    q, k, _ = p.on()
    gq, gk = p.dq.to(DEV), p.dk.to(DEV)
    want, ref = p.forward(), p.backward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fab().qk_rope(q, k, pos, freqs, stream=s, **kw)
    grads = fab().qk_rope_backward(gq, gk, pos, freqs, q=q, k=k, stream=s, **kw)
    s.synchronize()
    for a, b in zip((*got, *grads), (*want, *ref)):
        assert torch.equal(a, b)


def test_threads_with_streams_of_their_own():
    problems = [Problem(500 + 7 * i, 8, 2, 128, 128, norm="qk", seed=20 + i) for i in range(3)]
    refs = [(p.forward(), p.backward()) for p in problems]
    torch.cuda.synchronize()
    fails = []

    def work(p, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = (*p.forward(), *p.backward())
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, (*ref[0], *ref[1])))
        except Exception as e:   # noqa: BLE001
            fails.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(problems, refs)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not fails, fails


# ------------------------------------------------------------------ together
def test_training_step_through_the_rotation():
    """Projection outputs -> norm and rotation -> attention, and back: the
    gradients of the projections and of the norms' weights against the chain of
    the 64-bit definitions."""
    import oracle
    T, H, Hkv, d = 256, 4, 2, 64
    p = Problem(T, H, Hkv, d, d, norm="qk", seed=30, far=T)
    cu = np.array([0, 100, 256], dtype=np.int32)
    p.pos = torch.cat([torch.arange(100), torch.arange(156)]).int()
    scale, dev = d ** -0.5, torch.from_numpy(cu).to(DEV)
    q, k, v = (t.contiguous() for t in p.on())
    pos, freqs, kw = p.args()
    do = torch.randn(T, H, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    rq, rk = fab().qk_rope(q, k, pos, freqs, **kw)
    o, m, l = fab().forward_stats(rq, rk, v, dev, dev, cu, cu, True, scale)
    gq, gk, gv = fab().backward(rq, rk, v, o, do.to(DEV), m, l, dev, dev, cu, cu, True, scale)
    dq, dk, dqw, dkw = fab().qk_rope_backward(gq, gk, pos, freqs, q=q, k=k, **kw)
    # 64 bits from the rounded rotated rows on, so that the parts' own tests bound the difference
    dup = lambda t: np.repeat(f64(t), H // Hkv, 1)  # noqa: E731
    o64, m64, l64 = oracle.forward_packed(f64(rq), dup(rk), dup(v), cu, cu, scale, True)
    wq, wk = oracle.backward_packed(f64(rq), dup(rk), dup(v), o64, f64(do), m64, l64, cu, cu, scale, True)[:2]
    wk = wk.reshape(T, Hkv, H // Hkv, d).sum(2)
    for n, got, got_w, g in (("q", dq, dqw, wq), ("k", dk, dkw, wk)):
        ref, ref_w = rope.backward(g, f64(getattr(p, n)), p.pos.numpy(), p.theta, p.half, p.mscale, f64(p.w[n]), p.eps)
        for a, b in ((f64(got), ref), (f64(got_w), ref_w)):
            assert np.linalg.norm(a - b) <= 1e-2 * np.linalg.norm(b)


# ------------------------------------------------------------------ refusals
def test_refusals_that_need_a_device():
    p = Problem(8, 2, 2, 64, 64, norm="qk", seed=40)
    pos, freqs, kw = p.args()
    q, k, v = p.on()
    with pytest.raises(ValueError, match="positions is on cpu"):
        fab().qk_rope(q, k, pos.cpu(), freqs, **kw)
    with pytest.raises(fab().FabwdError, match="overlap"):
        fab().qk_rope(q, k, pos, freqs, out=(k, q), **kw)
    with pytest.raises(fab().FabwdError, match="rotary_dim"):
        fab().qk_rope(q, k, pos, fab().rope_freqs(72), **kw)
    with pytest.raises(fab().FabwdError, match="workspace"):
        fab().qk_rope_backward(q, k, pos, freqs, q=q, k=k, workspace=torch.zeros(8, device=DEV), **kw)
    with pytest.raises(fab().FabwdError, match="row_stride"):
        fab().qk_rope(q[:1].expand(8, 2, 64), None, pos, freqs)
