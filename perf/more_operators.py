"""Cases of the operators around attention: rotation of queries and keys by
their positions, with or without a norm per head (rope), its gradient
(rope_bwd), the same straight into the paged key-value cache (rope_append), and
attention of several new tokens per request over that cache (extend).

Every case runs in its plain form (elementary torch operations in 32 bits,
angles in 64) or, with ``own`` set, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one step of a serving loop: a row per request, long conversations; latency counts
        _rope("rope_decode_64", 64, 32, 8, 128, 128, "half", False, "none", 131072),
        # an odd number of rows, half of a small head rotated, neighbouring pairs, stretched positions
        _rope("rope_partial_8191", 8191, 16, 4, 64, 32, "interleaved", False, "linear", 32768),
        # a large packed training batch with a norm per head
        _rope("norm_rope_32k", 32768, 32, 8, 128, 128, "half", True, "parts", 8192),
        # the gradient of a training batch, a key/value head per query head
        _rope("norm_rope_bwd_16k", 16384, 16, 16, 128, 128, "half", True, "none", 4096, op="rope_bwd"),
        # the gradient at large heads of which a quarter is rotated, one key/value head, an odd number of rows
        _rope("norm_rope_bwd_d256", 5001, 8, 1, 256, 64, "interleaved", True, "none", 8192, op="rope_bwd"),
        # one step of a serving loop: a row per request, straight into the cache
        _append("rope_append_64", 64, 32, 8, 128, 128, "half", False, "none", 131072, 16, "bf16"),
        # a prompt batch with a norm per head enters an 8-bit cache
        _append("norm_rope_append_fp8", 8191, 32, 8, 128, 128, "half", True, "parts", 32768, 64, "fp8"),
        # a short question in one short conversation: latency counts
        _extend("extend_one_16", 1, 16, 16, 1024, 1024, 32, 8, 128, 16, 0, "bf16"),
        # a few drafted tokens per request are verified: bound by reading the cache
        _extend("extend_verify_64", 64, 1, 8, 256, 8192, 32, 8, 128, 16, 0, "bf16"),
        # chunks of long prompts behind what is cached of them already: bound by the products
        _extend("extend_chunk_4", 4, 2048, 2048, 0, 16384, 32, 8, 128, 64, 0, "bf16"),
        # ragged chunks and single tokens with a sliding window, odd page size and batch
        _extend("extend_window_d64", 37, 1, 700, 0, 5000, 16, 16, 64, 24, 1024, "bf16"),
        # large heads in an 8-bit cache, chunks and single tokens together
        _extend("extend_fp8_d256", 24, 1, 512, 0, 8192, 8, 2, 256, 32, 0, "fp8"),
    ]


def _rope(name, tokens, heads, heads_kv, dim, rotary, layout, norm, scaling, far, op="rope"):
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "heads_kv": heads_kv, "dim": dim,
            "rotary": rotary, "layout": layout, "norm": norm, "scaling": scaling, "far": far}


def _append(name, tokens, heads, heads_kv, dim, rotary, layout, norm, scaling, far, page, cache):
    case = _rope(name, tokens, heads, heads_kv, dim, rotary, layout, norm, scaling, far, op="rope_append")
    case.update(page=page, cache=cache)
    return case


def _extend(name, batch, new_lo, new_hi, lo, hi, heads, heads_kv, dim, page, window, cache):
    return {"name": name, "op": "extend", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "lo": lo, "hi": hi,
            "heads": heads, "heads_kv": heads_kv, "dim": dim, "page": page, "window": window, "cache": cache}


# products (new tokens * longest history and chunk * heads * dim) of the largest listed extend case
MOST_PRODUCTS = 4 * 2048 * 16384 * 32 * 128 // 2
# elements of the largest listed rope case's queries and keys
MOST_ELEMENTS = 32768 * 40 * 128


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "rope_append", "extend", "extend", "extend"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 64, 128, rng.randint(1, 130)])
    dim = rng.choice([64, 128, 128, 256])
    heads_kv = rng.choice([1, 2, 4, 8, 16])
    cache = rng.choice(["bf16", "fp8"])
    if op != "extend":
        heads = heads_kv * rng.choice([1, 2, 3, 4, 4, 5, 8])
        share = 2 if op == "rope" else 3
        most = max(64, min(32768, 2 * MOST_ELEMENTS // (share * (heads + 2 * heads_kv) * dim)))
        args = (_log(rng, 1, most), heads, heads_kv, dim, rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)]),
                rng.choice(["half", "half", "interleaved"]), rng.random() < 0.5,
                rng.choice(["none", "linear", "parts"]), _log(rng, 64, 1 << 20))
        case = _append("", *args, page, cache) if op == "rope_append" else _rope("", *args, op=op)
    else:
        heads = heads_kv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
        batch = _log(rng, 1, 128)
        unit = batch * heads * dim
        new = _log(rng, 1, max(1, min(4096, 32768 // batch, (1 << 28) // unit, math.isqrt(MOST_PRODUCTS // unit))))
        rows = MOST_PRODUCTS // (unit * new)
        held = (1 << 31) // (batch * heads_kv * dim)
        hi = _log(rng, 1, max(1, min(65536, rows - new, held - new)))
        lo = rng.choice([0, hi, _log(rng, 1, hi)])
        case = _extend("", batch, rng.choice([1, new]), new, lo, hi, heads, heads_kv, dim, page,
                       rng.choice([0, 0, 0, rng.randint(1, hi + new)]), cache)
    del case["name"]
    return case


def _spread(n, lo, hi):
    """n lengths from lo to hi: in equal ratios, in equal steps from 0."""
    at = [(i + 0.5) / n for i in range(n)]
    if lo >= 1:
        return [int(round(lo * (hi / lo) ** u)) for u in at]
    return [int(round(hi * u)) for u in at]


def _lengths(case, seed=0):
    """New tokens and cached tokens of every request: always the same pairs, in
    an order of the seed."""
    n = case["batch"]
    new, old = _spread(n, case["new_lo"], case["new_hi"]), _spread(n, case["lo"], case["hi"])
    paired = torch.randperm(n, generator=torch.Generator().manual_seed(n)).tolist()
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()
    return [new[i] for i in order], [old[paired[i]] for i in order]


def _size(case):
    return 1 if case["cache"] == "fp8" else 2


def work(case):
    heads, heads_kv, dim = case["heads"], case["heads_kv"], case["dim"]
    if case["op"] != "extend":
        tokens, norm = case["tokens"], case["norm"]
        row = (heads + heads_kv) * dim
        turned = (heads + heads_kv) * case["rotary"]
        if case["op"] == "rope":
            # a row in and out, its position; a product and a sum per rotated value twice, four steps of the norm
            return {"bytes": tokens * (4 * row + 4), "flops": tokens * (3 * turned + 4 * row * norm)}
        if case["op"] == "rope_bwd":
            return {"bytes": tokens * ((6 if norm else 4) * row + 4), "flops": tokens * (3 * turned + 10 * row * norm)}
        # position and slot (12), queries in and out, keys and values in and into the cache
        return {"bytes": tokens * (12 + 4 * heads * dim + 2 * heads_kv * dim * (2 + _size(case))),
                "flops": tokens * (3 * turned + 4 * row * norm)}
    pairs, keys = 0, 0
    window, new, old = case["window"], *_lengths(case)
    for n, s in zip(new, old):
        if window:
            free = max(0, min(n, window - s))   # rows that see less than a window
            pairs += free * s + free * (free + 1) // 2 + (n - free) * window
            keys += min(s + n, window + n - 1)
        else:
            pairs += n * s + n * (n + 1) // 2
            keys += s + n
    return {"bytes": 2 * keys * heads_kv * dim * _size(case) + sum(new) * heads * (4 * dim + 4)
            + 4 * (keys // case["page"]), "flops": 4 * pairs * heads * dim}


# ---------------------------------------------------------------- inputs
def _scaling(case):
    """factor, original length and factor of the outputs: positions divided by
    4; or divided by 4 only in the slow pairs, with the outputs grown."""
    if case["scaling"] == "linear":
        return 4.0, 0, 1.0
    if case["scaling"] == "parts":
        return 4.0, 4096, 0.1 * math.log(4.0) + 1.0
    return 1.0, 0, 1.0


def _cache(pool, case, gen):
    """A cache of normal values; 8-bit caches hold value / scale of the head."""
    shape = (pool, case["page"], case["heads_kv"], case["dim"])
    if case["cache"] == "bf16":
        return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen), None
    scale = 0.01 + 0.005 * torch.rand(case["heads_kv"], device=DEV, generator=gen)
    cache = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    rows = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, pool, rows):
        part = torch.empty((min(rows, pool - i),) + shape[1:], device=DEV).normal_(generator=gen)
        cache[i:i + rows] = (part / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return cache, scale


def _normal(shape, gen):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    heads, heads_kv, dim = case["heads"], case["heads_kv"], case["dim"]
    if case["op"] == "extend":
        return _prepare_extend(case, seed, gen)
    tokens = case["tokens"]
    factor, original, mscale = _scaling(case)
    state = {"op": case["op"], "layout": case["layout"], "rotary": case["rotary"], "mscale": mscale,
             "factor": factor, "original": original, "q_weight": None, "k_weight": None}
    # queries, keys and values are columns of one projection's output
    fused = _normal((tokens, heads + 2 * heads_kv, dim), gen)
    state.update(q=fused[:, :heads], k=fused[:, heads:heads + heads_kv])
    state["positions"] = torch.randint(0, case["far"], (tokens,), device=DEV, generator=gen, dtype=torch.int32)
    if case["norm"]:
        state["q_weight"], state["k_weight"] = (1 + 0.25 * _normal((dim,), gen) for _ in range(2))
    if case["op"] == "rope_bwd":
        state["dq"], state["dk"] = _normal((tokens, heads, dim), gen), _normal((tokens, heads_kv, dim), gen)
    if case["op"] == "rope_append":
        pool = -(-tokens // case["page"]) + 4
        state["v"] = fused[:, heads + heads_kv:]
        state["k_cache"], state["k_scale"] = _cache(pool, case, gen)
        state["v_cache"], state["v_scale"] = _cache(pool, case, gen)
        state["slots"] = torch.randperm(pool * case["page"], device=DEV, generator=gen)[:tokens]
    if own:
        import attention_backward_sm_gb300 as fab
        # a model's frequencies, made once
        state["freqs"] = fab.rope_freqs(case["rotary"], BASE, factor=factor, original_len=original, device=DEV)
        state["kind"] = fab.FA_ROPE_HALF if case["layout"] == "half" else fab.FA_ROPE_INTERLEAVED
    return state


def _prepare_extend(case, seed, gen):
    new, old = _lengths(case, seed)
    lens = [s + n for s, n in zip(old, new)]
    page = case["page"]
    have = [-(-s // page) for s in lens]
    pool = sum(have) + 4
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max(have)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    k_cache, k_scale = _cache(pool, case, gen)
    v_cache, v_scale = _cache(pool, case, gen)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {"op": "extend", "q": _normal((cu[-1], case["heads"], case["dim"]), gen), "k_cache": k_cache,
            "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale, "table": table.to(DEV),
            "seq": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "cu": torch.tensor(cu, dtype=torch.int32, device=DEV), "lens": lens, "ends": cu,
            "scale": case["dim"] ** -0.5, "window": case["window"]}


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if own:
        return _own(op, state)
    if op == "extend":
        return _plain_extend(state)
    turn = _plain_turns(state)
    if op == "rope":
        return {"q": _plain_rope(state, state["q"], state["q_weight"], turn).bfloat16(),
                "k": _plain_rope(state, state["k"], state["k_weight"], turn).bfloat16()}
    if op == "rope_bwd":
        out = {}
        for n in "qk":
            out["d" + n], out["d" + n + "_weight"] = _plain_rope_bwd(state, state["d" + n], state[n],
                                                                      state[n + "_weight"], turn)
        return out
    q = _plain_rope(state, state["q"], state["q_weight"], turn).bfloat16()
    k = _plain_rope(state, state["k"], state["k_weight"], turn)
    out = {"q": q}
    for n, x in (("k", k), ("v", state["v"].float())):
        cache, scale = state[n + "_cache"], state[n + "_scale"]
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448, 448)
        cache.view((-1,) + tuple(cache.shape[2:]))[state["slots"]] = x.to(cache.dtype)
        out[n + "_cache"] = cache
    return out


def _own(op, s):
    import attention_backward_sm_gb300 as fab
    if op == "extend":
        o, lse = fab.extend(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq"], s["cu"], s["scale"],
                            window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"o": o, "lse": lse}
    kw = dict(layout=s["kind"], mscale=s["mscale"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    if op == "rope":
        q, k = fab.qk_rope(s["q"], s["k"], s["positions"], s["freqs"], **kw)
        return {"q": q, "k": k}
    if op == "rope_bwd":
        dq, dk, dqw, dkw = fab.qk_rope_backward(s["dq"], s["dk"], s["positions"], s["freqs"], q=s["q"], k=s["k"], **kw)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    q = fab.qk_rope_append(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["k_cache"], s["v_cache"], s["slots"],
                           k_scale=s["k_scale"], v_scale=s["v_scale"], **kw)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_turns(s):
    """cos and sin [T, 1, rotary / 2] of the positions' angles, times mscale."""
    r = s["rotary"]
    f = BASE ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    if s["original"]:
        turns = s["original"] * f / (2 * math.pi)   # that the original length makes: few are slowed, many kept
        keep = ((turns - 1.0) / 31.0).clamp(0, 1)
        f = keep * f + (1 - keep) * f / s["factor"]
    else:
        f = f / s["factor"]
    a = s["positions"].double()[:, None] * f
    return tuple((s["mscale"] * x).float()[:, None] for x in (torch.cos(a), torch.sin(a)))


def _pairs(x, s):
    r = s["rotary"]
    if s["layout"] == "half":
        return x[..., :r // 2], x[..., r // 2:r]
    return x[..., 0:r:2], x[..., 1:r:2]


def _turned(x, s, cos, sin):
    a, b = _pairs(x, s)
    out = x.clone()
    to = _pairs(out, s)
    to[0].copy_(a * cos - b * sin)
    to[1].copy_(b * cos + a * sin)
    return out


def _plain_rope(s, x, weight, turn):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    return _turned(x, s, *turn)


def _plain_rope_bwd(s, dy, x, weight, turn):
    g = _turned(dy.float(), s, turn[0], -turn[1])
    if weight is None:
        return g.bfloat16(), None
    x = x.float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    x = x * inv
    d_weight = (g * x).sum((0, 1), dtype=torch.float64).float()
    g = g * weight.float()
    return (inv * (g - x * (g * x).mean(-1, keepdim=True))).bfloat16(), d_weight


def _plain_extend(s):
    q, cu = s["q"], s["ends"]
    tokens, heads, dim = q.shape
    page, heads_kv = s["k_cache"].shape[1:3]
    o = torch.zeros_like(q)
    lse = torch.full((tokens, heads), float("-inf"), device=DEV)
    for b, length in enumerate(s["lens"]):
        new = cu[b + 1] - cu[b]
        if not new:
            continue
        first = max(0, length - new - s["window"] + 1) if s["window"] else 0
        key = torch.arange(first, length, device=DEV)
        at = s["table"][b, key // page].long(), key % page
        k, v = s["k_cache"][at].float(), s["v_cache"][at].float()
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
        row = torch.arange(length - new, length, device=DEV)[:, None]
        seen = key <= row
        if s["window"]:
            seen &= key > row - s["window"]
        group = heads // heads_kv
        rows = q[cu[b]:cu[b + 1]].float().view(new, heads_kv, group, dim).permute(1, 2, 0, 3)
        x = torch.matmul(rows, k.permute(1, 2, 0)[:, None]) * s["scale"]
        x = torch.where(seen, x, float("-inf"))
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - top)
        total = x.sum(-1, keepdim=True)
        out = torch.matmul(x, v.transpose(0, 1)[:, None]) / total
        o[cu[b]:cu[b + 1]] = out.permute(2, 0, 1, 3).reshape(new, heads, dim).to(q.dtype)
        lse[cu[b]:cu[b + 1]] = (top + torch.log(total)).permute(2, 0, 1, 3).reshape(new, heads)
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(case, state)
    r, dim = case["rotary"], case["dim"]
    # the rotation as a product with complex numbers of the pairs
    theta = torch.tensor([_theta(case, i) for i in range(r // 2)], dtype=torch.float64, device=DEV)
    angle = torch.outer(state["positions"].double(), theta)[:, None]
    turn = torch.polar(torch.full_like(angle, _scaling(case)[2]), angle)
    half = case["layout"] == "half"

    def rotated(x, by):
        head = x[..., :r]
        z = torch.complex(head[..., :r // 2], head[..., r // 2:]) if half else \
            torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous())
        z = z * by
        back = torch.cat([z.real, z.imag], -1) if half else torch.view_as_real(z).flatten(-2)
        return torch.cat([back, x[..., r:]], -1)

    def unit(x):
        return x / torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / dim + EPS)

    if case["op"] == "rope_bwd":
        out = {}
        for n in "qk":
            g, w = rotated(state["d" + n].double(), turn.conj()), state[n + "_weight"]
            if w is None:
                out["d" + n], out["d" + n + "_weight"] = g, None
                continue
            x = state[n].double()
            u = unit(x)
            out["d" + n + "_weight"] = torch.einsum("thd,thd->d", g, u)
            g = g * w.double()
            # what is left of g when its part along x is taken out, with the length of x
            size = torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / dim + EPS)
            out["d" + n] = (g - u * torch.einsum("thd,thd->th", g, u)[..., None] / dim) / size
        return out
    done = {}
    for n in "qk":
        x, w = state[n].double(), state[n + "_weight"]
        done[n] = rotated(unit(x) * w.double() if w is not None else x, turn)
    if case["op"] == "rope":
        return done
    out = {"q": done["q"]}
    for n, x in (("k", done["k"]), ("v", state["v"].double())):
        cache, scale = state[n + "_cache"], state[n + "_scale"]
        flat = cache.double().view(-1, *cache.shape[2:])
        if scale is not None:
            # nearest multiple of the step of the value's power of two (3 fraction bits; 2^-9 near zero), ties to even
            x = x / scale.double()[:, None]
            power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
            step = torch.exp2(power - 3)
            x = (torch.round(x / step) * step).clamp(-448, 448)
        flat.index_copy_(0, state["slots"], x)
        out[n + "_cache"] = flat.view(cache.shape)
    return out


def _theta(case, i):
    """Angle per position of pair i."""
    factor, original, _ = _scaling(case)
    theta = math.pow(BASE, -2.0 * i / case["rotary"])
    if not original:
        return theta / factor
    wave = 2 * math.pi / theta
    ramp = min(1.0, max(0.0, (original / wave - 1.0) / (32.0 - 1.0)))
    return (1 - ramp) * theta / factor + ramp * theta


def _exact_extend(case, state):
    q = state["q"].double()
    heads, dim, heads_kv, page, window = case["heads"], case["dim"], case["heads_kv"], case["page"], case["window"]
    group, table, cu = heads // heads_kv, state["table"].long(), state["ends"]
    o = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=DEV)
    for b, n in enumerate(state["lens"]):
        rows = slice(cu[b], cu[b + 1])
        new = cu[b + 1] - cu[b]
        at = torch.arange(n, device=DEV)
        hidden = at[None] > at[n - new:, None]
        if window:
            hidden |= at[None] <= at[n - new:, None] - window
        pages = table[b, at // page]
        for h in range(heads_kv):
            k, v = (state[c][pages, at % page, h].double() for c in ("k_cache", "v_cache"))
            if state["k_scale"] is not None:
                k, v = k * state["k_scale"][h].double(), v * state["v_scale"][h].double()
            for g in range(h * group, (h + 1) * group):
                x = (q[rows, g] @ k.T * dim ** -0.5).masked_fill_(hidden, float("-inf"))
                lse[rows, g] = torch.logsumexp(x, -1)
                o[rows, g] = torch.softmax(x, -1) @ v
    return {"o": o, "lse": lse}
