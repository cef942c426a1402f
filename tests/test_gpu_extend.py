"""Attention of several new tokens per request over the paged cache, on the GPU
against the fp64 oracle.

Bounds per element (derived, not tuned), with u = 2^-8 (half a step of bf16 in
relation to the value) and fp32 sums that may truncate (2^-23 per addition):
  * a score of d products is off by at most delta = (d + 4) 2^-23 max|x|, |x| the
    sum of the absolute products, so every weight by 2 delta;
  * weights are rounded to w: 2^-8 (bf16) beside a bf16 cache, 2^-11 (fp16)
    beside an e4m3 one, and summed over n keys (n 2^-23); o is rounded to bf16:
    |o - ref| <= u |o| + (1 + 2^-6) (w + 2 delta + (n + 32) 2^-23) sum p |v| + f,
    f = n 2^-32 max|v| for fp16 weights (half their smallest step 2^-24 over the
    2^7 they are stored times; the row's reference key counts 1), else 0;
  * |lse - ref| <= 2 delta + (n + 32) 2^-23 + 2^-22 |lse|."""
import threading

import numpy as np
import pytest
import torch

import oracle
from oracle import paged, rope
from test_gpu_paged import strided

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def fab():
    import attention_backward_sm_gb300 as m
    return m


class Problem:
    """Requests of old cached and new tokens over randomly placed pages.  Slots
    past a request's last key and pages that nobody holds are NaN."""

    def __init__(self, old, new, heads, heads_kv, dim, page, kv="bf16", window=0, layout="plain", seed=0, q_scale=1.0,
                 pad=0, extra_width=1, bad=(), scale=None, freed=False):
        g = torch.Generator().manual_seed(seed)
        lens = [o + n for o, n in zip(old, new)]
        have = [-(-n // page) for n in lens]
        pool = sum(have) + 3
        order = torch.randperm(pool, generator=g)
        self.table = torch.full((len(lens), max(have + [0]) + extra_width), -1, dtype=torch.int32)
        shape = (pool, page, heads_kv, dim)
        k, v = torch.full(shape, float("nan")), torch.full(shape, float("nan"))
        at = 0
        for b, n in enumerate(lens):
            pages = order[at:at + have[b]]
            at += have[b]
            self.table[b, :have[b]] = pages.int()
            # with `freed`, nothing is left of what no row sees any more
            first = max(0, lens[b] - new[b] + 1 - window) if freed and window else 0
            j = torch.arange(first, n)
            if len(j):
                k[pages[j // page], j % page] = torch.randn(len(j), heads_kv, dim, generator=g)
                v[pages[j // page], j % page] = torch.randn(len(j), heads_kv, dim, generator=g)
            if freed and window:
                self.table[b, :first // page] = -1
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
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.q = (q_scale * torch.randn(sum(new) + pad, heads, dim, generator=g)).bfloat16()
        self.window, self.scale, self.layout = window, dim ** -0.5 if scale is None else scale, layout

    def device(self):
        on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        return dict(q=on(self.q), k_cache=strided(on(self.k), self.layout), v_cache=strided(on(self.v), self.layout),
                    block_table=on(self.table), seq_lens=on(self.lens), cu_new=on(self.cu), scale=self.scale,
                    window=self.window, k_scale=on(self.k_scale), v_scale=on(self.v_scale))

    def run(self, **kw):
        return fab().extend(**{**self.device(), **kw})

    def check(self, o, lse):
        ref, rlse, pv, xa, n = paged.extend(self.q.float(), self.k.float(), self.v.float(), self.table.numpy(),
                                            self.lens.numpy(), self.cu.numpy(), self.scale, self.window, self.k_scale,
                                            self.v_scale)
        o, lse = o.float().cpu().double().numpy(), lse.cpu().double().numpy()
        n = n[:, None]
        delta = (o.shape[-1] + 4) * 2.0 ** -23 * xa
        none = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(lse), none)
        assert np.all(o[none] == 0)
        rlse, lse = np.where(none, 0, rlse), np.where(none, 0, lse)
        tol = 2 * delta + (n + 32) * 2.0 ** -23 + 2.0 ** -22 * np.abs(rlse)
        assert np.all(np.abs(lse - rlse) <= tol), f"lse off by {np.abs(lse - rlse).max():.3e}"
        w = 2.0 ** -8 if self.k_scale is None else 2.0 ** -11
        tol = U * np.abs(ref) + (1 + 2.0 ** -6) * (w + 2 * delta + (n + 32) * 2.0 ** -23)[..., None] * pv
        if self.k_scale is not None:
            v = self.v.double() * self.v_scale.double()[:, None]
            tol = tol + (n * 2.0 ** -32)[..., None] * torch.nan_to_num(v).abs().max().item()
        bad = np.abs(o - ref) > tol + 1e-30
        assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.abs(o - ref)[bad].max():.3e}"


RAGGED_OLD, RAGGED_NEW = [0, 37, 300, 5, 0, 1000, 64], [1, 3, 130, 0, 200, 1, 65]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,heads_kv", [(1, 1), (6, 2), (8, 2), (5, 1), (16, 1)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_ragged_batch(dim, heads, heads_kv, kv):
    p = Problem(RAGGED_OLD, RAGGED_NEW, heads, heads_kv, dim, 16, kv, seed=dim + heads, pad=3)
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 7, 24, 64, 130, 400])
@pytest.mark.parametrize("layout", ["plain", "heads_first", "gaps"])
def test_pages_and_strides(page, layout, kv):
    p = Problem([0, 333, 128, 50], [70, 5, 128, 1], 4, 2, 128, page, kv, layout=layout, seed=page)
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 500, 5000])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sliding_window(dim, window, kv):
    p = Problem([0, 700, 129, 2000], [300, 40, 1, 77], 4, 2, dim, 24, kv, window=window, seed=window, freed=True)
    p.check(*p.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("old,new", [([0], [1]), ([0], [2]), ([127], [1]), ([128], [1]), ([127], [2]), ([63], [1]),
                                     ([64], [64]), ([0], [128]), ([0], [129]), ([0], [64]), ([255], [257])])
def test_borders_of_tiles(dim, old, new):
    for heads in (1, 3):
        p = Problem(old, new, heads, 1, dim, 16, seed=old[0] + new[0])
        p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("old,new,heads,heads_kv,dim", [
    ([30000], [3], 4, 1, 128),                       # one unit in nearly every run
    ([9000, 1, 20000], [1, 1, 1], 4, 2, 64),         # single tokens
    ([6000], [300], 8, 1, 128), ([5000], [70], 4, 4, 256), ([3000, 100, 4000], [200, 900, 1], 4, 2, 128),
    ([40] * 150, [2] * 150, 4, 2, 128),              # as many units as runs
    ([300] * 40, [5] * 40, 8, 8, 64)])
def test_units_in_several_runs(old, new, heads, heads_kv, dim, kv):
    p = Problem(old, new, heads, heads_kv, dim, 64, kv, seed=len(old))
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,heads_kv,dim", [(40, 2, 64), (24, 1, 128), (128, 1, 64), (130, 1, 128), (300, 1, 64),
                                                (144, 2, 256)])
def test_large_groups(heads, heads_kv, dim, kv):
    """Tiles that hold part of a token's heads, or several tokens and a part."""
    p = Problem([37, 300, 0], [5, 1, 9], heads, heads_kv, dim, 16, kv, seed=heads)
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("dim", [64, 256])
def test_costs_counted_coarsely(dim, window, kv):
    """Tables for 2^31 keys a request: costs count hundreds of keys at a time, so
    that those of full tables would fit, and cut the few blocks there are."""
    p = Problem([900, 0, 5, 2500] * 2, [20, 150, 1, 30] * 2, 8, 8, dim, 128, kv, window=window, seed=dim)
    p.check(*p.run())
    a = p.device()
    width, rows = 0x7fff0000 // 128, p.table.shape[1]
    flat = torch.full((width + 8 * rows,), -1, dtype=torch.int32, device=DEV)
    flat[:8 * rows] = a["block_table"].flatten()
    a["block_table"] = flat.as_strided((8, width), (rows, 1))   # entries past a request's own are not read
    p.check(*fab().extend(**a))
    fab().fa_check_device_status()


def test_many_requests():
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 4, 1300)]
    old = [int(x) for x in rng.integers(0, 60, 1300)]
    p = Problem(old, new, 4, 2, 64, 16, seed=5)
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_single_tokens_agree_with_decode(kv):
    lens = [1, 17, 300, 4000, 64]
    p = Problem([n - 1 for n in lens], [1] * 5, 8, 2, 128, 16, kv, seed=2)
    a = p.device()
    o, lse = fab().extend(**a)
    p.check(o, lse)
    a.pop("cu_new")
    o2, lse2 = fab().decode(**a)
    assert torch.all((lse - lse2).abs() <= 1e-4)
    assert torch.all((o.float() - o2.float()).abs() <= 0.05)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 256])
def test_missing_pages(dim, kv):
    """Entries that are no page, inside a tile, a whole tile and a whole request."""
    bad = [(0, 1, -1), (0, 3, 10 ** 6), (1, 0, -5)] + [(2, i, -1) for i in range(34)] + [(3, 20, 2 ** 31 - 1)]
    p = Problem([100, 3, 500, 400], [40, 10, 30, 1], 4, 2, dim, 16, kv, seed=7, bad=bad)
    p.check(*p.run())
    p = Problem([100], [40], 4, 2, dim, 16, kv, seed=7, bad=[(0, i, -1) for i in range(9)])
    o, lse = p.run()
    assert torch.all(o == 0) and torch.all(lse == float("-inf"))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30, 1e-3])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_scales(scale, kv):
    p = Problem([200, 10], [60, 5], 4, 2, 128, 16, kv, seed=9, scale=scale)
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_scale", [1e-25, 1e-6, 40.0])
def test_sizes_of_queries(q_scale, kv):
    """Scores that grow along the keys by far more than the reference's slack,
    and queries far from 1 (fp16 beside an e4m3 cache)."""
    p = Problem([900, 10], [60, 5], 4, 2, 128, 16, kv, seed=10, q_scale=q_scale)
    p.check(*p.run())
    p.q = p.q.abs()
    k = p.k.float()
    for b, n in enumerate(p.lens.tolist()):
        j = torch.arange(n)
        page = p.table[b, j // 16].long()
        k[page, j % 16] = (k[page, j % 16].abs() * (0.002 * j)[:, None, None]).clamp(max=448)
    p.k = k.to(p.k.dtype)
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("course", ["climb", "fall", "turns", "last", "first", "zigzag"])
def test_scores_far_apart(course, dim, kv):
    """Scores along the keys that a weight of 32 bits cannot hold beside each
    other, in every order: q . k = d a_j b with b the row's, a_j the key's."""
    p = Problem([700, 130, 40], [9, 200, 300], 6, 2, dim, 24, kv, seed=dim)
    base = p.k_scale.mean().item() * 448 if kv == "e4m3" else 8.0   # the most that a key may hold
    span = p.table.shape[1] * 24
    j = torch.arange(span)
    a = {"climb": j / 700 - 0.2, "fall": 0.8 - j / 700, "turns": torch.where(j // 70 % 2 == 0, 1.0, -1.0) * (j + 1) / 1000,
         "last": torch.where(j % 127 == 126, 1.0, -0.5), "first": torch.where(j == 0, 1.0, -0.5),
         "zigzag": torch.where(j % 2 == 0, 1.0, -1.0) * (j + 1) / 1000}[course] * base * 0.9
    scale = p.k_scale[:, None] if kv == "e4m3" else torch.ones(1)
    for b, n in enumerate(p.lens.tolist()):
        t = torch.arange(n)
        p.k[p.table[b, t // 24].long(), t % 24] = (a[t, None, None] / scale).clamp(-448, 448).expand(n, 2, dim).to(p.k.dtype)
    rows = torch.linspace(-12, 12, p.q.shape[0] * 6).reshape(-1, 6, 1)
    p.q = rows.expand(p.q.shape).bfloat16().contiguous()
    p.check(*p.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("climb", [0.03, 0.3, 3.0])
def test_large_values_behind_climbing_scores(climb, dim):
    """Values of up to 2^100 and scores that climb along the keys, slowly and by more
    than a block's slack: weights against an old reference do not carry the sums out
    of the range of 32 bits."""
    p = Problem([700, 130, 40], [9, 200, 300], 6, 2, dim, 24, seed=dim + 1, scale=1.0)
    span = p.table.shape[1] * 24
    j = torch.arange(span)
    for b, n in enumerate(p.lens.tolist()):
        t = torch.arange(n)
        at = p.table[b, t // 24].long(), t % 24
        p.k[at] = (climb * j[:n, None, None] / dim).expand(n, 2, dim).bfloat16()
        p.v[at] = (p.v[at].float().clamp(-4, 4) * 2.0 ** 98).bfloat16()
    p.q = torch.ones_like(p.q)
    p.check(*p.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 30])
def test_windows_before_the_first_key(window, dim, kv):
    """Requests with fewer keys than new tokens, whose first rows lie before all
    keys: no window, however wide, shifts what the others see."""
    p = Problem([0, 0, 90], [60, 200, 70], 4, 2, dim, 16, kv, seed=19, window=window)
    p.lens[0], p.lens[1], p.lens[2] = 50, 7, 40
    p.check(*p.run())


def test_a_padded_batch_of_a_million_requests():
    """Requests without tokens are no units, however many there are."""
    p = Problem([40, 3, 200], [3, 1, 2], 32, 32, 64, 16, seed=18, extra_width=0)
    want = p.run()
    a = p.device()
    batch = 1 << 20
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    lens[:2], lens[batch - 1] = a["seq_lens"][:2], a["seq_lens"][2]
    cu = torch.full((batch + 1,), 4, dtype=torch.int32, device=DEV)
    cu[:2], cu[batch] = a["cu_new"][:2], a["cu_new"][3]
    table = torch.full((batch, p.table.shape[1]), -1, dtype=torch.int32, device=DEV)
    table[:2], table[batch - 1] = a["block_table"][:2], a["block_table"][2]
    a.update(seq_lens=lens, cu_new=cu, block_table=table)
    o, lse = fab().extend(**a)
    fab().fa_check_device_status()
    p.check(o, lse)
    assert o.shape == want[0].shape


def test_lengths_that_do_not_fit():
    """Lengths below 0 and below the number of new tokens (their first rows see
    nothing), past the table, and a request cut off by the rows of q."""
    p = Problem([50, 0, 100, 30], [20, 30, 12, 40], 4, 2, 128, 16, seed=11, extra_width=3)
    p.lens[0], p.lens[1], p.lens[2] = -7, 12, 5000
    p.q = p.q[:80]
    p.table[2, 7:] = p.table[2, 0]   # past its own pages: keys that are there
    p.check(*p.run())


def test_nothing_to_do():
    p = Problem([5, 6], [0, 0], 4, 2, 64, 16, seed=12, pad=9)
    o, lse = p.run()
    assert o.shape == (9, 4, 64) and torch.all(o == 0) and torch.all(lse == float("-inf"))
    p = Problem([5, 6], [0, 0], 4, 2, 64, 16, seed=12)
    o, lse = p.run()
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    a = Problem([5], [3], 4, 2, 64, 16, seed=12).device()
    a.update(block_table=a["block_table"][:0], seq_lens=a["seq_lens"][:0], cu_new=a["cu_new"][:1])
    o, lse = fab().extend(**a)
    assert torch.all(o == 0) and torch.all(lse == float("-inf"))
    p = Problem([5], [3], 4, 2, 64, 16, seed=12)
    a = p.device()
    a.update(k_cache=a["k_cache"][:0], v_cache=a["v_cache"][:0])
    o, lse = fab().extend(**a)
    assert torch.all(o == 0) and torch.all(lse == float("-inf"))


def test_outputs_of_the_caller_and_strided_queries():
    p = Problem([100, 300], [40, 3], 8, 2, 128, 16, seed=13)
    want = p.run()
    a = p.device()
    fused = torch.full((43, 12, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    fused[:, :8] = a["q"]
    a["q"] = fused[:, :8]
    o = torch.full((43, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    work = torch.full((fab().fa_extend_workspace_size(128),), 255, dtype=torch.uint8, device=DEV)
    got, none = fab().extend(**a, out=(o, None), workspace=work)
    assert none is None and got.data_ptr() == o.data_ptr() and torch.equal(o, want[0])
    lse = torch.empty(43, 8, device=DEV)
    fab().fa_extend(o=o, lse=lse, **a)
    assert torch.equal(lse, want[1])


def test_offsets_past_32_bits():
    """Pages so far apart that most lie past 2^31 elements."""
    p = Problem([300], [40], 4, 2, 128, 16, seed=14)
    want = p.run()
    a = p.device()
    pages, stride = p.k.shape[0], 1 << 28
    big = torch.empty(pages * stride, dtype=torch.bfloat16, device=DEV)
    for i, n in enumerate(("k_cache", "v_cache")):
        t = big.as_strided(p.k.shape, (stride, 2 * 128, 128, 1), i << 16)
        t.copy_(a[n])
        a[n] = t
    got = fab().extend(**a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ repeated, captured, at once
def test_same_bits_again():
    p = Problem(RAGGED_OLD, RAGGED_NEW, 8, 2, 128, 16, seed=15)
    a = p.device()
    first = fab().extend(**a)
    for _ in range(20):
        got = fab().extend(**a)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    fab().fa_check_device_status()


def test_captured_with_lengths_that_change():
    """A captured call takes the lengths, offsets and pages that the buffers hold
    at the replay; two graphs have a workspace each from their pools."""
    one = Problem([700, 40, 0], [30, 1, 60], 8, 2, 128, 16, seed=16, extra_width=60)
    two = Problem([10, 1500, 300], [1, 80, 10], 8, 2, 128, 16, seed=17, extra_width=10)
    a, b = one.device(), two.device()
    fab().extend(**a)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for args in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fab().extend(**args))
        graphs.append(g)
    for _ in range(2):
        for g, out, p in zip(graphs, outs, (one, two)):
            out[0].fill_(3)
            g.replay()
            p.check(*out)
    # the first graph with other lengths: fewer keys of the same pages
    one.lens -= torch.tensor([300, 0, 20], dtype=torch.int32)
    a["seq_lens"].copy_(one.lens)
    graphs[0].replay()
    one.check(*outs[0])


def test_threads_with_streams_of_their_own():
    problems = [Problem([500 + 100 * i, 30], [90, 1], 8, 2, 128, 16, seed=20 + i) for i in range(3)]
    args = [p.device() for p in problems]
    refs = [fab().extend(**a) for a in args]
    torch.cuda.synchronize()
    fails = []

    def work(a, ref):
        try:
            s = torch.cuda.Stream()
            for _ in range(30):
                got = fab().extend(**a, stream=s)
            s.synchronize()
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        except Exception as e:   # noqa: BLE001
            fails.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(args, refs)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not fails, fails


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_prompts_in_chunks_then_tokens(kv):
    """A serving loop: prompts enter in chunks of uneven sizes (plan, rotation
    with norms into the cache, attention over it), then single tokens; all rows
    against the 64-bit definition from the projections on."""
    H, Hkv, d, page, scale = 4, 2, 64, 8, 64 ** -0.5
    g = torch.Generator().manual_seed(30)
    steps = [[50, 7, 0], [1, 33, 20], [64, 1, 1], [1, 1, 1], [3, 1, 5]]
    total = [sum(s[b] for s in steps) for b in range(3)]
    x = [torch.randn(n, H + 2 * Hkv, d, generator=g).bfloat16() for n in total]
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    sc = None if kv == "bf16" else torch.full((Hkv,), 0.02)
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    pages = 40
    kc, vc = (torch.full((pages, page, Hkv, d), float("nan"), device=DEV).to(dt) for _ in range(2))
    i32 = dict(dtype=torch.int32, device=DEV)
    table, lens, start = torch.full((3, 20), -1, **i32), torch.zeros(3, **i32), torch.zeros(1, **i32)
    free = torch.randperm(pages, generator=g).int().to(DEV)
    freqs = fab().rope_freqs(d)
    kw = {} if sc is None else dict(k_scale=sc.to(DEV), v_scale=sc.to(DEV))
    done, got = [0, 0, 0], [[], [], []]
    for s in steps:
        rows = torch.cat([x[b][done[b]:done[b] + s[b]] for b in range(3)]).to(DEV)
        pad = torch.zeros(2, H + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
        rows = torch.cat([rows, pad])
        plan = fab().kv_plan(table, lens, torch.tensor(s, **i32), free, page, len(rows), free_start=start)
        q = fab().qk_rope_append(rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:], plan.positions, freqs, kc, vc,
                                 plan.slots, q_weight=wq.to(DEV), k_weight=wk.to(DEV), **kw)
        o, lse = fab().extend(q, kc, vc, table, plan.seq_lens, plan.cu_new, scale, **kw)
        assert torch.all(o[-2:] == 0) and torch.all(lse[-2:] == float("-inf"))
        lens, start = plan.seq_lens, plan.free_next
        at = 0
        for b in range(3):
            got[b].append(o[at:at + s[b]].float().cpu())
            at += s[b]
            done[b] += s[b]
    theta = rope.frequencies(d)
    for b in range(3):
        n = total[b]
        f = x[b].double().numpy()
        q64 = rope.forward(f[:, :H], np.arange(n), theta, True, 1.0, wq, 1e-6)
        k64 = rope.forward(f[:, H:H + Hkv], np.arange(n), theta, True, 1.0, wk, 1e-6)
        v64 = f[:, H + Hkv:]
        out = torch.cat(got[b]).double().numpy()
        for h in range(H):
            ref = oracle.forward_head(q64[:, h], k64[:, h // 2], v64[:, h // 2], scale, True, 0)[0]
            err = np.linalg.norm(out[:, h] - ref) / np.linalg.norm(ref)
            # bf16: q, k, the weights and o rounded, 2^-8 at most each; e4m3: k and v by 2^-4
            assert err <= (2.0 ** -6 if kv == "bf16" else 2.0 ** -3), err


def test_refusals_that_need_a_device():
    p = Problem([40], [8], 4, 2, 128, 16, seed=40)
    a = p.device()
    for over, word in [(dict(seq_lens=a["seq_lens"].cpu()), "seq_lens is on cpu"), (dict(cu_new=a["cu_new"][:1]), "cu_new"),
                       (dict(q=a["q"].float()), "q must be"), (dict(out=(a["q"][:, :2], None)), "o must be"),
                       (dict(out=(torch.empty_like(a["q"]), torch.empty(8, 3, device=DEV))), "lse")]:
        with pytest.raises(ValueError, match=word):
            fab().extend(**{**a, **over})
    for over, code, word in [(dict(out=(a["q"], None)), 1, "overlap"), (dict(window=-1), 1, "window"),
                             (dict(scale=float("nan")), 1, "scale"),
                             (dict(workspace=torch.zeros(16, device=DEV)), 1, "workspace")]:
        with pytest.raises(fab().FabwdError, match=word) as e:
            fab().extend(**{**a, **over})
        assert e.value.code == code
