"""Paged cache operators on the GPU against the fp64 oracle.

Bounds for decode, per element (derived, not tuned): with u the unit
roundoff of a stored type (bf16: 2^-8) and fp32 sums that may truncate
(2^-23 per addition),
  * a score of d products is off by at most delta = (d + 4) 2^-23 max|x|,
    |x| the sum of the absolute products, so every weight by 2 delta;
  * weights are rounded to w (fp16 for e4m3 caches: 2^-11; two bf16 numbers:
    2^-16) and summed over n keys (n 2^-23), o is rounded to bf16 (u |o|):
    |o - ref| <= u |o| + (1 + 2^-6) (w + 2 delta + (n + 32) 2^-23) sum p |v| + f
    with f = n 2^-29 max|v| for fp16 weights, whose steps below 2^-14 are
    2^-24, half of that off, over the 2^4 that the weight of a row's
    reference key (which counts 1 in the sum) is stored with; else 0;
  * |lse - ref| <= 2 delta + (n + 32) 2^-23 + 2^-22 |lse|.
plan and append move whole numbers and bits: they are compared exactly."""
import threading

import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from oracle import paged
from paged_paths import PATHS

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def fab():
    import attention_backward_sm_gb300 as m
    return m


def strided(cache, layout):
    """The same [pages, page, Hkv, d] contents in another memory layout."""
    if layout == "heads_first":
        return cache.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "gaps":   # every second page and padded slots of a larger buffer
        p, s, h, d = cache.shape
        big = torch.full((p, 2, s, h + 1, d), 1.0).to(cache.dtype).to(cache.device)
        big[:, 1, :, :h] = cache
        return big[:, 1, :, :h]
    return cache


class Problem:
    """Requests of given lengths over randomly placed pages.  Slots past a
    request's last key and pages that nobody holds are NaN."""

    def __init__(self, lens, heads, heads_kv, dim, page, kv="bf16", window=0, layout="plain", seed=0, q_scale=1.0,
                 extra_width=1, bad=()):
        g = torch.Generator().manual_seed(seed)
        have = [-(-n // page) for n in lens]
        width = max(have + [0]) + extra_width
        pool = sum(have) + 3
        order = torch.randperm(pool, generator=g)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        shape = (pool, page, heads_kv, dim)
        k = torch.full(shape, float("nan"))
        v = torch.full(shape, float("nan"))
        for b, n in enumerate(lens):
            pages = order[at:at + have[b]]
            at += have[b]
            self.table[b, :have[b]] = pages.int()
            if n:
                j = torch.arange(n)
                k[pages[j // page], j % page] = torch.randn(n, heads_kv, dim, generator=g)
                v[pages[j // page], j % page] = torch.randn(n, heads_kv, dim, generator=g)
        for b, i, entry in bad:
            self.table[b, i] = entry
        self.k_scale = self.v_scale = None
        if kv == "e4m3":
            self.k_scale = 0.01 + 0.01 * torch.rand(heads_kv, generator=g)
            self.v_scale = 0.01 + 0.01 * torch.rand(heads_kv, generator=g)
            k = (k / self.k_scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            v = (v / self.v_scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            k, v = k.bfloat16(), v.bfloat16()
        self.k, self.v = k, v
        self.q = (q_scale * torch.randn(len(lens), heads, dim, generator=g)).bfloat16()
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.window, self.scale, self.layout = window, dim ** -0.5, layout

    def device(self):
        kc, vc = strided(self.k.to(DEV), self.layout), strided(self.v.to(DEV), self.layout)
        on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        return dict(q=on(self.q), k_cache=kc, v_cache=vc, block_table=on(self.table), seq_lens=on(self.lens),
                    scale=self.scale, window=self.window, k_scale=on(self.k_scale), v_scale=on(self.v_scale))

    def run(self, **kw):
        return fab().decode(**{**self.device(), **kw})

    def check(self, o, lse, rows=None):
        ref, rlse, pv, xa = paged.decode(self.q.float(), self.k.float(), self.v.float(), self.table.numpy(),
                                         self.lens.numpy(), self.scale, self.window,
                                         self.k_scale, self.v_scale)
        o, lse = o.float().cpu().double().numpy(), lse.cpu().double().numpy()
        d = o.shape[-1]
        n = self.lens.clamp(min=0).numpy()[:, None]
        if self.window:
            n = np.minimum(n, self.window)
        delta = (d + 4) * 2.0 ** -23 * xa
        none = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(lse), none)
        assert np.all(o[none] == 0)
        rlse, lse = np.where(none, 0, rlse), np.where(none, 0, lse)
        tol = 2 * delta + (n + 32) * 2.0 ** -23 + 2.0 ** -22 * np.abs(rlse)
        assert np.all(np.abs(lse - rlse) <= tol), f"lse off by {np.abs(lse - rlse).max():.3e}"
        w = 2.0 ** -16 if self.k_scale is None else 2.0 ** -11
        tol = U * np.abs(ref) + (1 + 2.0 ** -6) * (w + 2 * delta + (n + 32) * 2.0 ** -23)[..., None] * pv
        if self.k_scale is not None:
            v = self.v.double() * self.v_scale.double()[:, None]
            tol = tol + (n * 2.0 ** -29)[..., None] * torch.nan_to_num(v).abs().max().item()
        bad = np.abs(o - ref) > tol + 1e-30
        assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.abs(o - ref)[bad].max():.3e}"


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("batch,page,seq_hi,new_hi,width,free,pad,start", [
    (1, 16, 0, 1, 4, 8, 0, 0), (3, 1, 5, 4, 16, 64, 3, 2), (64, 16, 500, 1, 40, 80, 0, 0),
    (257, 7, 90, 3, 20, 300, 10, 5), (1000, 64, 0, 130, 4, 3100, 7, 0), (5, 16, 40, 60, 5, 9, 0, 0),
    (1, 8, 3, 20000, 2600, 2600, 1, 0), (300, 16, 33, 0, 4, 0, 2, 0)])
def test_plan_matches_the_oracle(batch, page, seq_hi, new_hi, width, free, pad, start):
    rng = np.random.default_rng(batch * 1000 + page)
    seq = rng.integers(0, seq_hi + 1, batch)
    new = rng.integers(0, new_hi + 1, batch)
    if batch > 2:
        seq[1], new[2] = -4, -1          # lengths below 0 count as 0
    table = np.full((batch, width), -1)
    pages = rng.permutation(batch * width + free)
    for b in range(batch):
        have = min(-(-max(seq[b], 0) // page), width)
        table[b, :have] = pages[b * width:b * width + have]
    free_pages = pages[batch * width:]
    tokens = int(np.maximum(new, 0).sum()) + pad
    want = paged.plan(table, seq, new, free_pages, page, tokens, start)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    wide = i32(np.concatenate([table, np.full((batch, 3), 77)], 1))   # rows further apart than they are long
    args = (wide[:, :width], i32(seq), i32(new), i32(free_pages))
    for call in range(2):                                             # the second changes nothing
        got = fab().kv_plan(*args, page, tokens, free_start=i32([start]))
        torch.cuda.synchronize()
        for name, g, w in zip(("table", "slots", "positions", "cu_new", "seq_lens", "free_next"),
                              (args[0], *got), (*want[:5], np.array([want[5]]))):
            assert np.array_equal(g.cpu().numpy(), w), (name, call)
        assert torch.all(wide[:, width:] == 77)


def test_plan_too_few_slots_keeps_the_count():
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.full((2, 4), -1, **i32)
    p = fab().kv_plan(table, torch.zeros(2, **i32), torch.tensor([5, 3], **i32), torch.arange(8, **i32), 4, 6)
    assert p.slots.tolist() == [0, 1, 2, 3, 4, 8] and p.cu_new.tolist() == [0, 5, 8] and p.free_next.tolist() == [3]


@pytest.mark.parametrize("tokens", [0, 1, 4, 5, 7, 8, 16, 17, 18, 29, 30, 31, 40, 41, 200])
@pytest.mark.parametrize("start,free", [(0, 30), (3, 30), (0, 6), (2, 0)])
def test_plan_too_few_slots_enters_every_page(tokens, start, free):
    """Cuts at num_tokens before, inside and after requests with several new
    pages (held pages, rows too short and an empty list among them): the table
    and the tokens' places are those of the definition, and a second call with
    slots for all tokens finds its pages in the table."""
    page, seq, new = 4, [0, 3, 8, 0, 5, 0, 1], [5, 12, 0, 1, 11, 40, 2]
    width = 6
    table = np.full((len(seq), width), -1)
    at = 50
    for b, n in enumerate(seq):
        for i in range(-(-n // page)):
            table[b, i], at = at, at + 1
    free_pages = np.random.default_rng(7).permutation(free)
    want = paged.plan(table, seq, new, free_pages, page, tokens, start)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    wide = i32(np.concatenate([table, np.full((len(seq), 2), 77)], 1))
    for call in range(2):
        got = fab().kv_plan(wide[:, :width], i32(seq), i32(new), i32(free_pages), page, tokens, free_start=i32([start]))
        for name, g, w in zip(("table", "slots", "positions", "cu_new", "seq_lens", "free_next"),
                              (wide[:, :width], *got), (*want[:5], np.array([want[5]]))):
            assert np.array_equal(g.cpu().numpy(), w), (name, call)
        assert torch.all(wide[:, width:] == 77)


def test_plan_too_few_slots_for_many_requests():
    """More requests than threads and pages than a block takes at once, lengths
    past the table's rows (a thousand million tokens) among them."""
    rng = np.random.default_rng(8)
    batch, page, width = 3000, 16, 40
    seq, new = rng.integers(0, 300, batch), rng.integers(0, 300, batch)
    table = np.full((batch, width), -1)
    for b, n in enumerate(seq):
        table[b, :-(-n // page)] = 10 ** 6 + b
    free_pages = rng.permutation(batch * width)
    want = paged.plan(table, seq, new, free_pages, page, 1000)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    got_table = i32(table)
    got = fab().kv_plan(got_table, i32(seq), i32(new), i32(free_pages), page, 1000)
    for g, w in zip((got_table, *got), (*want[:5], np.array([want[5]]))):
        assert np.array_equal(g.cpu().numpy(), w)
    new[:] = 10 ** 9
    got_table = i32(table)
    fab().kv_plan(got_table, i32(seq), i32(new), i32(free_pages), page, 10)
    held = -(-seq // page)
    first = np.cumsum(width - held) - (width - held)
    got_table = got_table.cpu().numpy()
    for b in range(batch):
        assert np.array_equal(got_table[b, held[b]:], free_pages[first[b]:first[b] + width - held[b]])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("tokens,heads_kv,dim,page", [(1, 1, 64, 16), (7, 8, 128, 16), (333, 3, 64, 5), (129, 2, 256, 64)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["plain", "heads_first", "gaps"])
def test_append_writes_named_slots_only(tokens, heads_kv, dim, page, kv, layout):
    g = torch.Generator().manual_seed(tokens)
    pool = -(-tokens // page) + 3
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    bits = torch.int16 if kv == "bf16" else torch.uint8
    fused = (30 * torch.randn(tokens, 5 + 2 * heads_kv, dim, generator=g)).bfloat16()
    fused[0, 5, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30])
    fused[-1, -1, :3] = torch.tensor([-0.0, 1e-30, 448.5])
    k, v = fused[:, 5:5 + heads_kv], fused[:, 5 + heads_kv:]
    slots = torch.randperm(pool * page, generator=g)[:tokens]
    if tokens > 3:
        slots[1], slots[3] = -1, pool * page       # skipped
    scale = None if kv == "bf16" else 0.05 + torch.rand(heads_kv, generator=g)
    before = torch.randn(pool, page, heads_kv, dim, generator=g).to(dtype)
    kc, vc = strided(before.to(DEV), layout), strided(before.clone().to(DEV), layout)
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    dev = fused.to(DEV)
    fab().kv_append(dev[:, 5:5 + heads_kv], dev[:, 5 + heads_kv:], kc, vc, slots.to(DEV), on(scale), on(scale))
    ok = (slots >= 0) & (slots < pool * page)
    for got, new in ((kc, k), (vc, v)):
        want = before.clone().view(bits).view(-1, heads_kv, dim)
        row = new if scale is None else (new.float() / scale[:, None]).clamp(-448, 448).to(dtype)
        want[slots[ok]] = row.contiguous().view(bits)[ok]
        got, want = got.cpu().contiguous().view(dtype), want.view(dtype).view(before.shape)
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan)
        assert torch.equal(got.view(bits)[~nan], want.view(bits)[~nan])


@pytest.mark.parametrize("scale", [1.0, 0.05, 3.0, 1 / 3, 0.0123456, 2.0 ** -7, 448.0, 1e-30, 1e30, 1e-40, 3e38])
def test_append_rounds_every_bf16_value_as_the_quotient(scale):
    """All 65536 bf16 bit patterns: the 8-bit value of the fp32 quotient, bit
    for bit (values next to a border of two 8-bit numbers among them)."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(-1, 1, 64)
    s = torch.tensor([scale])
    want = (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)
    kc = torch.zeros(len(x) // 16, 16, 1, 64, dtype=torch.float8_e4m3fn, device=DEV)
    vc = torch.zeros_like(kc)
    fab().kv_append(x.to(DEV), x.to(DEV), kc, vc, torch.arange(len(x), device=DEV), s.to(DEV), s.to(DEV))
    for got in (kc, vc):
        got = got.cpu().view(want.shape)
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan)
        assert torch.equal(got.view(torch.uint8)[~nan], want.view(torch.uint8)[~nan])


@pytest.mark.parametrize("scale", [None, 2.0 ** -100, 2.0 ** -30, 0.0625, 0.5, 1.0, 8.0, 2.0 ** 100, 2.0 ** -101, 2.0 ** 101])
def test_append_rounds_every_bf16_value_by_a_power_of_two(scale):
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(-1, 1, 64)
    want = (x.float() / (1.0 if scale is None else scale)).clamp(-448, 448).to(torch.float8_e4m3fn)
    kc = torch.zeros(len(x) // 16, 16, 1, 64, dtype=torch.float8_e4m3fn, device=DEV)
    vc = torch.zeros_like(kc)
    s = None if scale is None else torch.tensor([scale], device=DEV)
    fab().kv_append(x.to(DEV), x.to(DEV), kc, vc, torch.arange(len(x), device=DEV), s, s)
    for got in (kc, vc):
        got = got.cpu().view(want.shape)
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan)
        assert torch.equal(got.view(torch.uint8)[~nan], want.view(torch.uint8)[~nan])


def test_append_without_a_scale_does_not_divide():
    """Values on the border of two 8-bit numbers, of which a scale of 1 has many,
    cost nothing: no more than 1.3 times the time of a scale that has none (with
    a division per value it was 1.7)."""
    heads_kv, dim, page, tokens, calls = 8, 128, 64, 32768, 20
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(tokens, heads_kv, dim, device=DEV, generator=g).bfloat16() for _ in range(2))
    kc = torch.zeros(tokens // page, page, heads_kv, dim, dtype=torch.float8_e4m3fn, device=DEV)
    vc = torch.zeros_like(kc)
    slots = torch.randperm(tokens, device=DEV, generator=g)
    scales = [torch.full((heads_kv,), 0.0123, device=DEV), None, torch.full((heads_kv,), 0.25, device=DEV)]
    best = [float("inf")] * 3
    for rep in range(8):
        for i, s in enumerate(scales):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(2_000_000)   # the calls are queued behind it: the GPU's time alone
            a.record()
            for _ in range(calls):
                fab().kv_append(k, v, kc, vc, slots, s, s)
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    assert max(best[1:]) <= 1.3 * best[0], best


@pytest.mark.parametrize("tokens,heads_kv,dim", [(3000, 40, 64), (257, 9, 256), (5000, 1, 64)])
def test_append_many_rows_and_wide_rows(tokens, heads_kv, dim):
    """Rows of more and of fewer pieces than a block has threads."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    k, v = (torch.randn(tokens, heads_kv, dim, device=DEV, generator=g).bfloat16() for _ in range(2))
    kc = torch.zeros(-(-tokens // 7), 7, heads_kv, dim, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    slots = torch.randperm(kc.shape[0] * 7, device=DEV, generator=g)[:tokens]
    fab().kv_append(k, v, kc, vc, slots)
    for got, new in ((kc, k), (vc, v)):
        want = torch.zeros_like(got).view(-1, heads_kv, dim)
        want[slots] = new
        assert torch.equal(got.view_as(want), want)


# ------------------------------------------------------------------ decode
# query and key/value heads: 1 to 16 to a key/value head and more (in chunks),
# key/value heads that go by 4, by 2 or one at a time
GROUPS = [(1, 1), (4, 4), (8, 2), (6, 2), (14, 2), (9, 1), (16, 1), (20, 1), (40, 1), (12, 12), (20, 4), (32, 4),
          (44, 4), (64, 4), (32, 2), (18, 6), (27, 1), (33, 1), (48, 2)]


# wide: a block table long enough for tiles of several key/value heads, which
# calls with few keys at most do not take
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads,heads_kv", GROUPS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_head_layouts(heads, heads_kv, dim, kv, wide):
    p = Problem([1, 0, 63, 64, 65, 130, 300], heads, heads_kv, dim, 16, kv, seed=heads * dim,
                extra_width=8000 if wide else 1)
    p.check(*p.run())


@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 256])
@pytest.mark.parametrize("window", [0, 1, 17, 64, 1000])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads_kv,wide", [(2, False), (4, True)])
def test_decode_pages_and_windows(page, window, kv, heads_kv, wide):
    p = Problem([1, page, page + 1, 127, 128, 129, 517, 0, 16], 4, heads_kv, 128, page, kv, window, seed=page + window,
                extra_width=1 + (100_000 // page if wide else 0))
    p.check(*p.run())


@pytest.mark.parametrize("layout", ["plain", "heads_first", "gaps"])
@pytest.mark.parametrize("dim,kv", [(64, "bf16"), (128, "e4m3"), (256, "bf16")])
@pytest.mark.parametrize("heads,heads_kv,width", [(6, 3, 1), (8, 4, 8000)])
def test_decode_layouts_and_strided_queries(layout, dim, kv, heads, heads_kv, width):
    p = Problem([200, 33, 1, 90], heads, heads_kv, dim, 16, kv, layout=layout, seed=dim, extra_width=width)
    fused = torch.full((4, 12, dim), float("nan"), dtype=torch.bfloat16)
    fused[:, :heads] = p.q
    p.check(*p.run(q=fused.to(DEV)[:, :heads]))


@pytest.mark.parametrize("batch,hi,heads,heads_kv,dim,kv", [
    (1, 20000, 8, 2, 128, "bf16"),        # one request over every SM
    (1, 9000, 1, 1, 64, "e4m3"),
    (1, 30000, 4, 4, 64, "bf16"),         # one head group over every SM
    (2, 12000, 8, 8, 128, "e4m3"),
    (300, 90, 4, 4, 64, "bf16"),          # many more requests than SMs
    (700, 40, 4, 1, 64, "e4m3"),
    (33, 3000, 4, 1, 256, "bf16"),        # ragged
    (40, 2500, 24, 1, 128, "e4m3")])
def test_decode_splits(batch, hi, heads, heads_kv, dim, kv):
    lens = [int(x) for x in np.random.default_rng(batch).integers(0, hi + 1, batch)]
    lens[0] = hi
    for width in (1, 20000):
        p = Problem(lens, heads, heads_kv, dim, 16, kv, seed=batch, extra_width=width)
        o, lse = p.run()
        p.check(o, lse)
        again = p.run()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("path", PATHS, ids=str)
def test_decode_paths(path):
    """Every way of cutting and joining runs, with each shape of tiles (what a
    case takes is pinned in test_paged_cpu.py).  The workspace holds NaN before
    the call, and what lies behind it is left alone."""
    f = fab()
    have = -(-max(path.lens) // path.page)
    p = Problem(path.lens, path.heads, path.heads_kv, path.dim, path.page, path.kv, seed=path.heads,
                extra_width=path.width - have)
    size = f.fa_decode_workspace_size(path.batch, path.heads, path.heads_kv, path.dim)
    work = torch.full((size + 4096,), 255, dtype=torch.uint8, device=DEV)
    args = p.device()
    o, lse = f.decode(**args, workspace=work[:size])
    assert torch.all(work[size:] == 255)
    p.check(o, lse)
    again = f.decode(**args)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_peaked_growing_and_shrinking_scores(kv):
    """Weights on a few keys; the running maximum rises or falls all along."""
    for q_scale in (30.0, 0.0):
        p = Problem([700, 129], 4, 2, 128, 16, kv, q_scale=q_scale, seed=9)
        p.check(*p.run())
    for sign in (1, -1):
        p = Problem([640, 640], 4, 1, 128, 16, seed=10)
        ramp = torch.linspace(-4, 4, 640) * sign
        j = torch.arange(640)
        for b in range(2):
            p.k[p.table[b].long()[j // 16], j % 16, 0, 0] = ramp.bfloat16()
        p.q[..., 0] = 40.0
        p.check(*p.run())


def test_decode_bad_pages_are_not_seen():
    for heads_kv, width in ((2, 1), (4, 8000)):
        p = Problem([70, 200, 40, 10], 4, heads_kv, 128, 16, seed=12, extra_width=width,
                    bad=[(0, 1, -1), (0, 4, 10 ** 9), (1, 0, -7), (1, 12, 2 ** 31 - 1), (3, 0, -1)])
        o, lse = p.run()
        p.check(o, lse)
        assert torch.all(o[3] == 0) and torch.all(lse[3] == -float("inf"))


def test_decode_lengths_are_clamped_to_the_table():
    p = Problem([32, 20, 5], 4, 2, 64, 16, extra_width=0, seed=13)
    p.lens[0], p.lens[2] = 2 ** 31 - 1, -3
    o, lse = p.run()
    p.lens[0], p.lens[2] = 32, 0
    p.check(o, lse)


def test_decode_visible_nan_and_inf_reach_the_output():
    """A NaN key or value that is seen shows, in its request and head only."""
    for kv in ("bf16", "e4m3"):
        p = Problem([50, 50], 4, 2, 64, 16, kv, seed=14)
        clean = p.run()
        nan = torch.tensor(float("nan")).to(p.k.dtype)
        p.v[p.table[0, 1].long(), 3, 0, 5] = nan
        p.k[p.table[1, 0].long(), 2, 1, 7] = nan
        o, lse = p.run()
        assert torch.isnan(o[0, :2, 5]).all() and torch.isnan(o[1, 2:]).all() and torch.isnan(lse[1, 2:]).all()
        assert torch.equal(o[0, 2:], clean[0][0, 2:]) and torch.equal(o[1, :2], clean[0][1, :2])
        assert torch.equal(lse[0], clean[1][0])
    # -inf scores beside finite ones weigh nothing, wherever they come first
    for at in (0, 49):
        p = Problem([50], 1, 1, 64, 16, seed=15)
        p.q[..., 0] = 1.0
        p.k[p.table[0, at // 16].long(), at % 16, 0, 0] = -float("inf")
        o, lse = p.run()
        keep = [j for j in range(50) if j != at]
        k = torch.stack([p.k[p.table[0, j // 16].long(), j % 16, 0] for j in keep]).double()
        want = torch.logsumexp(p.scale * (k @ p.q[0, 0].double()), 0)
        assert abs(lse.item() - want.item()) < 1e-4 and torch.isfinite(o).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,heads_kv,dim,width", [(4, 2, 64, 1), (8, 1, 128, 1), (4, 4, 128, 8000), (4, 4, 64, 8000),
                                                      (12, 6, 128, 4000)])
def test_decode_weights_are_not_rounded_to_16_bits(heads, heads_kv, dim, width, kv):
    """Up to 8 query heads to a key/value head (of at most 128 at e4m3): values
    that cancel, so that o is small beside sum p |v| and its own rounding does not
    hide that of the weights.  A weight is two 16-bit numbers; fp16: the upper
    11 bits, exact, and a rest below 2^-10 of it, rounded to 2^-11 of itself
    (2^-21), or to steps of 2^-24 where it is subnormal (2^-25 over the 2^4 that
    weights carry)."""
    lens = [2, 4, 6, 9, 40]
    p = Problem(lens, heads, heads_kv, dim, 16, kv, seed=dim, q_scale=0.02, extra_width=width)
    for b, n in enumerate(lens):
        for j in range(n):
            p.v[p.table[b, j // 16].long(), j % 16] = torch.tensor((-1.0) ** j * 384).to(p.v.dtype)
    o, lse = p.run()
    ref, _, pv, xa = paged.decode(p.q.float(), p.k.float(), p.v.float(), p.table.numpy(), p.lens.numpy(), p.scale, 0,
                                  p.k_scale, p.v_scale)
    n = p.lens.numpy()[:, None]
    delta = (dim + 4) * 2.0 ** -23 * xa
    w = 2.0 ** -16 if kv == "bf16" else 2.0 ** -21
    tol = U * np.abs(ref) + (1 + 2.0 ** -6) * (w + 2 * delta + (n + 32) * 2.0 ** -23)[..., None] * pv
    if kv == "e4m3":
        tol = tol + (n * 2.0 ** -29)[..., None] * 384 * p.v_scale.max().item()
    off = np.abs(o.float().cpu().double().numpy() - ref)
    assert np.all(off <= tol), (off / tol).max()
    p.check(o, lse)


@pytest.mark.parametrize("heads,heads_kv,dim,width", [(4, 2, 64, 1), (4, 4, 128, 8000), (16, 1, 128, 1), (8, 1, 256, 1),
                                                      (24, 1, 64, 1), (16, 8, 128, 8000)])
def test_decode_visible_infinite_values(heads, heads_kv, dim, width):
    """An infinite value among those a row sees makes its element infinite, as
    any weight above zero times it is; two of both signs make it NaN; the
    others are the definition's.  Requests of one key (a weight of exactly 1),
    of part of a tile, of several tiles and of several blocks' runs."""
    lens = [1, 20, 200, 6000]
    p = Problem(lens, heads, heads_kv, dim, 16, seed=dim + heads, extra_width=width)
    want = torch.zeros(len(lens), heads_kv, dim)
    for b, n in enumerate(lens):
        for i, j in enumerate({0, n // 3, n - 1}):
            for h in range(heads_kv):
                for col, value in ((3 * i, float("inf")), (3 * i + 1, -float("inf")), (dim - 1, (-1) ** i * float("inf"))):
                    p.v[p.table[b, j // 16].long(), j % 16, h, col] = value
                    want[b, h, col] = want[b, h, col] + value
    o, lse = p.run()
    got = o.float().cpu().view(len(lens), heads_kv, -1, dim)
    want = want[:, :, None].expand(got.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    infinite = torch.isinf(want)
    assert torch.equal(got[infinite], want[infinite])
    p.v = torch.nan_to_num(p.v, nan=float("nan"), posinf=0.0, neginf=0.0)
    ref = paged.decode(p.q.float(), p.k.float(), p.v.float(), p.table.numpy(), p.lens.numpy(), p.scale)[0]
    special = infinite.view(o.shape) | torch.isnan(want).reshape(o.shape)
    p.check(torch.where(special.to(DEV), torch.from_numpy(ref).to(DEV).bfloat16(), o), lse)


def test_decode_empty_table_and_no_lse():
    f = fab()
    p = Problem([3, 0], 4, 2, 64, 16, seed=15)
    d = p.device()
    for none in ({"block_table": d["block_table"][:, :0]},
                 {"k_cache": d["k_cache"][:0], "v_cache": d["v_cache"][:0]}):
        o, lse = f.decode(**{**d, **none})
        assert torch.all(o == 0) and torch.all(lse == -float("inf"))
    full, _ = f.decode(**d)
    o = torch.empty_like(full)
    ws = torch.empty(max(1, f.fa_decode_workspace_size(2, 4, 2, 64)), dtype=torch.uint8, device=DEV)
    f.fa_decode(d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["seq_lens"], o, None, p.scale, workspace=ws)
    assert torch.equal(o, full)
    o, lse = f.decode(**{**d, "q": d["q"][:0], "block_table": d["block_table"][:0], "seq_lens": d["seq_lens"][:0]})
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kv):
    """A cache of 2^31 + some elements: pages behind the 2^31st element are
    written and read at their own place."""
    f = fab()
    page, heads_kv, dim = 64, 8, 128
    pool = (1 << 31) // (page * heads_kv * dim) + 4
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    kc = torch.empty(pool, page, heads_kv, dim, dtype=dtype, device=DEV)
    vc = torch.empty_like(kc)
    p = Problem([150, 64], 8, heads_kv, dim, page, kv, seed=16)
    where = torch.tensor([pool - 1, 0, pool - 2, 1, pool - 3, pool // 2, pool - 4, 2])[:p.k.shape[0]]
    table = torch.where(p.table >= 0, where[p.table.clamp(min=0).long()].int(), -1)
    for src, dst in ((p.k, kc), (p.v, vc)):
        dst[where.to(DEV)] = src.to(DEV)
    d = p.device()
    small = f.decode(**d)
    big = f.decode(**{**d, "k_cache": kc, "v_cache": vc, "block_table": table.to(DEV)})
    assert torch.equal(small[0], big[0]) and torch.equal(small[1], big[1])
    row = torch.randn(1, heads_kv, dim, device=DEV).bfloat16()
    slot = torch.tensor([(pool - 1) * page + 5], device=DEV)
    f.kv_append(row, row, kc, vc, slot)
    assert torch.equal(kc[pool - 1, 5].float(), row[0].to(dtype).float())


@pytest.mark.parametrize("heads,dim,code,word", [(4, 96, 2, "head_dim"), (3, 64, 1, "multiple"), (0, 64, 1, "multiple"),
                                                 (2050, 64, 2, "1024")])
def test_decode_raises_the_code_of_the_c_entry(heads, dim, code, word):
    f = fab()
    i32 = dict(dtype=torch.int32, device=DEV)
    cache = torch.zeros(4, 16, 2, dim, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(1, heads, dim, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(f.FabwdError, match=word) as e:
        f.decode(q, cache, cache, torch.zeros(1, 1, **i32), torch.ones(1, **i32), 0.1)
    assert e.value.code == code
    if dim == 96:
        with pytest.raises(f.FabwdError, match=word) as e:
            f.kv_append(cache[0, :1], cache[0, :1], cache, cache.clone(), torch.zeros(1, dtype=torch.int64, device=DEV))
        assert e.value.code == code


# ------------------------------------------------------------------ as a program uses them
def test_prefill_then_decode_steps_match_the_forward():
    """plan -> append -> forward over the prompts, then plan -> append ->
    decode token by token: every step's row is the row that the packed causal
    forward over all tokens gives (both within their bounds of the oracle)."""
    f = fab()
    H, Hkv, d, page, steps = 8, 2, 128, 16, 20
    prompt, B = [37, 1, 64, 15], 4
    total = [n + steps for n in prompt]
    case = si.Case("serve", H, d, total, total, True, 77, heads_kv=Hkv)
    q, k, v, _ = (t.to(DEV) for t in case.tensors())
    cu = torch.from_numpy(case.cu_q).to(DEV)
    full_o, full_lse = f.forward_lse(q, k, v, cu, cu, case.cu_q, case.cu_q, True, case.softmax_scale)
    kc = torch.full((64, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = torch.full_like(kc, float("nan"))
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.full((B, 8), -1, **i32)
    free = torch.randperm(64, generator=torch.Generator().manual_seed(1)).int().to(DEV)
    seq, start = torch.zeros(B, **i32), torch.zeros(1, **i32)
    base = case.cu_q[:-1]
    rows = np.concatenate([base[b] + np.arange(n) for b, n in enumerate(prompt)])
    for step in range(steps + 1):
        if step:
            rows = np.array([base[b] + n + step - 1 for b, n in enumerate(prompt)])
        at = torch.from_numpy(rows).to(DEV)
        new = torch.tensor(prompt if step == 0 else [1] * B, **i32)
        plan = f.kv_plan(table, seq, new, free, page, len(rows), free_start=start)
        f.kv_append(k[at], v[at], kc, vc, plan.slots)
        seq, start = plan.seq_lens, plan.free_next
        last = at if step else torch.from_numpy(np.array([base[b] + n - 1 for b, n in enumerate(prompt)])).to(DEV)
        o, lse = f.decode(q[last], kc, vc, table, seq, case.softmax_scale)
        torch.testing.assert_close(lse, full_lse[last], rtol=2e-6, atol=1e-5)
        # each side is within 2^-8 (|o| + sum p|v|) of the exact row; sum p|v| < 4 for these values
        assert (o.float() - full_o[last].float()).abs().max().item() <= 2 * U * 8
    assert start.item() == sum(-(-n // page) for n in total)
    flat = kc.view(-1, Hkv, d)
    for b, n in enumerate(total):
        j = torch.arange(n, device=DEV)
        slots = table[b].long()[j // page] * page + j % page
        assert torch.equal(flat[slots], k[int(base[b]):int(base[b]) + n])


def test_decode_loop_in_a_graph():
    """One captured step (plan, append, decode, state copied forward) replayed:
    the same as eager steps, while another graph with its own buffers replays
    on a second stream."""
    f = fab()
    H, Hkv, d, page, B, steps = 8, 2, 64, 16, 3, 40

    class Loop:
        def __init__(self, seed):
            g = torch.Generator(device=DEV).manual_seed(seed)
            i32 = dict(dtype=torch.int32, device=DEV)
            rnd = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
            self.qs, self.ks, self.vs = rnd(steps, B, H, d), rnd(steps, B, Hkv, d), rnd(steps, B, Hkv, d)
            self.q, self.k, self.v = rnd(B, H, d), rnd(B, Hkv, d), rnd(B, Hkv, d)
            self.kc, self.vc = rnd(16, page, Hkv, d), rnd(16, page, Hkv, d)
            self.table, self.seq, self.start = torch.full((B, 4), -1, **i32), torch.zeros(B, **i32), torch.zeros(1, **i32)
            self.new = torch.ones(B, **i32)
            self.free = torch.arange(16, **i32)

        def feed(self, i):
            self.q.copy_(self.qs[i]), self.k.copy_(self.ks[i]), self.v.copy_(self.vs[i])

        def step(self):
            p = f.kv_plan(self.table, self.seq, self.new, self.free, page, B, free_start=self.start)
            f.kv_append(self.k, self.v, self.kc, self.vc, p.slots)
            out = f.decode(self.q, self.kc, self.vc, self.table, p.seq_lens, d ** -0.5)
            self.seq.copy_(p.seq_lens), self.start.copy_(p.free_next)
            return out

        def reset(self):
            self.table.fill_(-1), self.seq.zero_(), self.start.zero_()

    loops = [Loop(1), Loop(2)]
    want = []
    for lp in loops:
        got = []
        for i in range(steps):
            lp.feed(i)
            got.append(tuple(t.clone() for t in lp.step()))
        want.append(got)
        lp.reset()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for lp in loops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lp.step())
        graphs.append(g)
        lp.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in loops]
    got = [[], []]
    for i in range(steps):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                loops[n].feed(i)
                graphs[n].replay()
                got[n].append(tuple(t.clone() for t in outs[n]))
    torch.cuda.synchronize()
    for n in range(2):
        for a, b in zip(want[n], got[n]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_from_two_threads_on_two_streams():
    """Calls in flight at once, each with its own workspace, give the bits of
    a plain call; each caller's stream is ordered after its own."""
    f = fab()
    p = Problem([900, 5, 333, 64], 8, 2, 128, 16, seed=21)
    args = p.device()
    plain = f.decode(**args)
    p.check(*plain)
    torch.cuda.synchronize()
    results, errors = {}, []

    def worker(tid):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                results[tid] = [f.decode(**args) for _ in range(30)]
            stream.synchronize()
        except Exception as e:  # reported on the main thread
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for got in results.values():
        for o, lse in got:
            assert torch.equal(o, plain[0]) and torch.equal(lse, plain[1])


def test_stream_argument():
    """stream=: the work runs on it, after what is queued there."""
    f = fab()
    p = Problem([100, 40], 4, 2, 64, 16, seed=22)
    args = p.device()
    plain = f.decode(**args)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    late = args["q"].clone().zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(10_000_000)
        late.copy_(args["q"])
    o, lse = f.decode(**{**args, "q": late}, stream=stream)
    stream.synchronize()
    assert torch.equal(o, plain[0]) and torch.equal(lse, plain[1])


def test_stream_argument_keeps_the_inputs():
    """Inputs dropped right after a call on another stream: their memory is
    not reused before that stream has read them."""
    f = fab()
    p = Problem([300, 40], 4, 2, 64, 16, seed=23)
    plain = p.run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    args = p.device()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(50_000_000)
    o, lse = f.decode(**args, stream=stream)
    sizes = [(t.shape, t.dtype) for t in args.values() if torch.is_tensor(t)]
    del args
    junk = [torch.full(s, 1.0, device=DEV).to(d) for s, d in sizes for _ in range(3)]
    stream.synchronize()
    assert torch.equal(o, plain[0]) and torch.equal(lse, plain[1])
    assert len(junk) == 3 * len(sizes)


def test_refusals_beside_a_device():
    """Malformed outputs and workspaces, tensors and streams of other devices:
    refused before anything is launched."""
    f = fab()
    p = Problem([40, 3], 4, 2, 64, 16, seed=31)
    a = p.device()
    o, lse = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 4, device=DEV)
    wide = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV)

    class Elsewhere:
        stream_id, device_index, device_type = 0, torch.cuda.current_device() + 1, 1

    for kw, word in ((dict(out=o), "tuple"), (dict(out=(o,)), "tuple"), (dict(out=[o, lse]), "tuple"),
                     (dict(out=(o.float(), lse)), "o must"), (dict(out=(o[:1], lse)), "o must"),
                     (dict(out=(wide[:, :4], lse)), "contiguous"), (dict(out=(o, lse.double())), "lse"),
                     (dict(out=(o, lse[:, :3])), "lse"), (dict(out=(o, wide)), "lse"), (dict(out=(None, lse)), "o must"),
                     (dict(out=(o.cpu(), lse)), "o is on"), (dict(out=(o, lse.cpu())), "lse is on"),
                     (dict(workspace=torch.zeros(2, 1 << 20, device=DEV).t()), "workspace"),
                     (dict(workspace=torch.zeros(1 << 20)), "workspace is on"),
                     (dict(seq_lens=a["seq_lens"].cpu()), "seq_lens is on"), (dict(v_cache=a["v_cache"].cpu()), "v_cache is on"),
                     (dict(stream=Elsewhere()), "stream is on device")):
        with pytest.raises(ValueError, match=word):
            f.decode(**{**a, **kw})
    with pytest.raises(f.FabwdError, match="workspace"):
        f.decode(**a, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(f.FabwdError, match="overlap"):
        f.decode(**a, out=(a["q"], lse))
    with pytest.raises(AttributeError):
        f.decode(**a, stream="a stream")
    i32 = dict(dtype=torch.int32, device=DEV)
    args = (a["block_table"], a["seq_lens"], torch.ones(2, **i32), torch.arange(4, **i32), 16)
    out = [torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(2, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32),
           torch.zeros(1, **i32)]
    for i, word in enumerate(("slots", "positions", "cu_new", "seq_lens_out", "free_next")):
        with pytest.raises(ValueError, match=word):   # another type
            f.fa_kv_plan(*args, *(out[:i] + [out[i].float()] + out[i + 1:]))
        with pytest.raises(ValueError, match=word):   # another device
            f.fa_kv_plan(*args, *(out[:i] + [out[i].cpu()] + out[i + 1:]))
    with pytest.raises(ValueError, match="positions"):
        f.fa_kv_plan(*args, *(out[:1] + [out[2]] + out[2:]))
    with pytest.raises(f.FabwdError, match="seq_lens_out"):
        f.fa_kv_plan(*args, *(out[:3] + [a["seq_lens"]] + out[4:]))
    slots = torch.zeros(2, dtype=torch.int64, device=DEV)
    rows = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    for kw, word in ((dict(k=rows.cpu()), "k is on"), (dict(slots=slots.cpu()), "slots is on"),
                     (dict(stream=Elsewhere()), "stream is on device"), (dict(k_scale=torch.ones(2)), "k_scale is on")):
        with pytest.raises(ValueError, match=word):
            f.kv_append(**{**dict(k=rows, v=rows, k_cache=a["k_cache"], v_cache=a["v_cache"], slots=slots), **kw})
    got, want = f.decode(**a), p.run()   # the device is as it was
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_serving_steps_match_the_definition(kv):
    """plan -> append -> decode, prompts and then token by token, one request
    getting none for some steps: tables, slots, caches and rows are the
    definition's over the same history (rows within their bounds)."""
    f = fab()
    H, Hkv, d, page, pool, width = 8, 2, 128, 16, 40, 8
    g = torch.Generator().manual_seed(41)
    p = Problem([1] * 4, H, Hkv, d, page, kv, seed=41)
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    bits = torch.int16 if kv == "bf16" else torch.uint8
    p.k = torch.full((pool, page, Hkv, d), float("nan")).to(dtype)
    p.v = p.k.clone()
    kc, vc = p.k.to(DEV), p.v.to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    free = torch.randperm(pool, generator=g).int()
    table, seq, start = torch.full((4, width), -1, **i32), torch.zeros(4, **i32), torch.zeros(1, **i32)
    want_table, want_seq, nxt = np.full((4, width), -1), [0] * 4, 0
    for step in range(14):
        new = [37, 0, 64, 15] if step == 0 else [1, 1, 1, 1 if step % 3 else 0]
        n = sum(new) + 2                       # two rows of padding
        want_table, slots, _, _, after, nxt = paged.plan(want_table, want_seq, new, free.numpy(), page, n, nxt)
        want_seq = after.tolist()
        rows = [torch.randn(n, Hkv, d, generator=g).bfloat16() for _ in range(2)]
        plan = f.kv_plan(table, seq, torch.tensor(new, **i32), free.to(DEV), page, n, free_start=start)
        f.kv_append(rows[0].to(DEV), rows[1].to(DEV), kc, vc, plan.slots, on(p.k_scale), on(p.v_scale))
        seq, start = plan.seq_lens, plan.free_next
        assert np.array_equal(table.cpu().numpy(), want_table) and np.array_equal(plan.slots.cpu().numpy(), slots)
        ok = torch.from_numpy(slots >= 0)
        for cache, row, scale, got in ((p.k, rows[0], p.k_scale, kc), (p.v, rows[1], p.v_scale, vc)):
            if scale is not None:
                row = (row.float() / scale[:, None]).clamp(-448, 448).to(dtype)
            cache.view(bits).view(-1, Hkv, d)[torch.from_numpy(slots)[ok]] = row.view(bits)[ok]
            assert torch.equal(got.cpu().view(bits), cache.view(bits))
        p.q = torch.randn(4, H, d, generator=g).bfloat16()
        p.table, p.lens = torch.from_numpy(want_table), torch.tensor(want_seq, dtype=torch.int32)
        p.check(*f.decode(p.q.to(DEV), kc, vc, table, seq, p.scale, k_scale=on(p.k_scale), v_scale=on(p.v_scale)))


def test_strides_that_are_never_used_do_not_matter():
    """Of a dimension of one, and of tensors without elements."""
    f = fab()
    i32 = dict(dtype=torch.int32, device=DEV)
    p = Problem([40, 3], 4, 1, 64, 16, seed=51)          # one key/value head: laid out alike, whatever its stride
    a = p.device()
    v = a["v_cache"].as_strided(a["v_cache"].shape, (16 * 64, 64, 1 << 20, 1))
    got = f.decode(**{**a, "v_cache": v})
    p.check(*got)
    rows = torch.randn(5, 1, 64, device=DEV).bfloat16()
    caches = [torch.zeros_like(v), torch.zeros(v.shape, dtype=v.dtype, device=DEV).as_strided(v.shape, v.stride())]
    f.kv_append(rows, rows, *caches, torch.arange(5, device=DEV))
    assert torch.equal(caches[0], caches[1]) and torch.equal(caches[0].view(-1, 64)[:5], rows[:, 0])
    empty = torch.zeros(0, 6, **i32).as_strided((0, 6), (0, 0))
    plan = f.kv_plan(empty, torch.zeros(0, **i32), torch.zeros(0, **i32), torch.arange(4, **i32), 16, 3,
                     free_start=torch.tensor([2], **i32))
    assert plan.slots.tolist() == [-1] * 3 and plan.positions.tolist() == [0] * 3
    assert plan.cu_new.tolist() == [0] and plan.seq_lens.numel() == 0 and plan.free_next.tolist() == [2]
    o, lse = f.decode(a["q"][:0].as_strided((0, 4, 64), (0, 0, 0)), a["k_cache"], v, empty, a["seq_lens"][:0], p.scale)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    f.kv_append(rows[:0].as_strided((0, 1, 64), (0, 0, 0)), rows[:0], *caches, torch.zeros(0, dtype=torch.int64, device=DEV))
