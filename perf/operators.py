"""Cases of the paged key-value cache operators: building block tables and
slot maps (plan), writing new keys and values into the cache (append) and
attention of one new token per request over the cache (decode).

Every case runs in its plain form (elementary torch operations in 32 bits)
or, with ``own`` set, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one step of a serving loop: each request gets one token, some a new page
        _plan("plan_decode_64", 64, 256, 8192, 1, 1, 16),
        # the same with a large number of short conversations
        _plan("plan_decode_2048", 2048, 1, 4096, 1, 1, 16),
        # prompts of very different lengths enter an empty cache at once
        _plan("plan_prefill_32", 32, 0, 0, 256, 8192, 64),
        # one step of a serving loop: one row per request, out of a fused projection
        _append("append_decode_64", 64, 32, 8, 128, 16, "bf16"),
        # a prompt batch enters the cache
        _append("append_prefill_32k", 32768, 32, 8, 128, 64, "bf16"),
        # an odd number of rows into an 8-bit cache of small heads
        _append("append_fp8_d64", 8191, 16, 16, 64, 16, "fp8"),
        # a single short conversation: latency counts
        _decode("decode_one_1k", 1, 1024, 1024, 32, 8, 128, 16, 0, "bf16"),
        # a serving batch of ragged lengths
        _decode("decode_gqa_64", 64, 256, 8192, 32, 8, 128, 16, 0, "bf16"),
        # few very long documents: the cache's length has to be split
        _decode("decode_long_4", 4, 65536, 131072, 32, 8, 128, 64, 0, "bf16"),
        # sliding window, a key/value head per query head, odd page size and batch
        _decode("decode_window_d64", 37, 1, 5000, 16, 16, 64, 24, 1024, "bf16"),
        # the largest batch, from an 8-bit cache
        _decode("decode_fp8_128", 128, 1024, 16384, 32, 8, 128, 64, 0, "fp8"),
        # large heads, all query heads on one key/value head
        _decode("decode_mqa_d256", 16, 512, 8192, 8, 1, 256, 32, 0, "bf16"),
    ]


def _plan(name, batch, lo, hi, new_lo, new_hi, page):
    return {"name": name, "op": "plan", "batch": batch, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi,
            "page": page}


def _append(name, tokens, heads, heads_kv, dim, page, cache):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads, "heads_kv": heads_kv, "dim": dim,
            "page": page, "cache": cache}


def _decode(name, batch, lo, hi, heads, heads_kv, dim, page, window, cache):
    return {"name": name, "op": "decode", "batch": batch, "lo": lo, "hi": hi, "heads": heads, "heads_kv": heads_kv,
            "dim": dim, "page": page, "window": window, "cache": cache}


# rows of keys (padded to the longest request) * heads_kv * dim of the largest listed decode case
MOST_DECODE = 128 * 16384 * 8 * 128


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 64, 128, rng.randint(1, 130)])
    if op == "plan":
        hi = _log(rng, 1, 16384)
        case = _plan("", _log(rng, 1, 4096), 0, 0, 1, 1, page)
        if rng.random() < 0.5:
            case.update(lo=rng.randint(0, hi), hi=hi)
        else:
            new = min(_log(rng, 1, 16384), max(1, (1 << 19) // case["batch"]))
            case.update(lo=0, hi=rng.choice([0, hi]), new_lo=rng.randint(0, new), new_hi=new)
    elif op == "append":
        dim = rng.choice([64, 128, 256])
        heads_kv = rng.choice([1, 2, 4, 8, 16])
        most = (32768 * 8 * 128) // (heads_kv * dim)
        case = _append("", _log(rng, 1, min(most, 65536)), heads_kv * rng.choice([1, 2, 4, 8]), heads_kv, dim, page,
                       rng.choice(["bf16", "fp8"]))
    else:
        dim = rng.choice([64, 128, 128, 256])
        heads_kv = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12, 16, 32])
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(131072, MOST_DECODE // (batch * heads_kv * dim * max(1, group // 4)))))
        lo = rng.choice([0, hi, _log(rng, 1, hi)])
        window = rng.choice([0, 0, 0, rng.randint(1, hi)])
        case = _decode("", batch, lo, hi, heads_kv * group, heads_kv, dim, page, window, rng.choice(["bf16", "fp8"]))
    del case["name"]
    return case


def _spread(n, lo, hi):
    """n lengths from lo to hi: in equal ratios, in equal steps from 0."""
    at = [(i + 0.5) / n for i in range(n)]
    if lo >= 1:
        return [int(round(lo * (hi / lo) ** u)) for u in at]
    return [int(round(hi * u)) for u in at]


def _lengths(case, lo="lo", hi="hi"):
    return _spread(case["batch"], case[lo], case[hi])


def work(case):
    if case["op"] == "plan":
        seq, new, page = _lengths(case), _lengths(case, "new_lo", "new_hi"), case["page"]
        pages = sum(-(-(s + n) // page) - -(-s // page) for s, n in zip(seq, new))
        # per request: two lengths in, length and offset out; per new page: read and write of its number;
        # per token: slot (8) and position (4)
        return {"bytes": 16 * case["batch"] + 8 * pages + 12 * sum(new), "flops": 0}
    if case["op"] == "append":
        row = case["heads_kv"] * case["dim"]
        return {"bytes": case["tokens"] * (2 * row * (2 + _size(case)) + 8), "flops": 0}
    keys = sum(min(n, case["window"]) if case["window"] else n for n in _lengths(case))
    heads, dim = case["heads"], case["dim"]
    return {"bytes": 2 * keys * case["heads_kv"] * dim * _size(case) + case["batch"] * heads * (4 * dim + 4)
            + 4 * (keys // case["page"]), "flops": 4 * keys * heads * dim}


def _size(case):
    return 1 if case["cache"] == "fp8" else 2


# ---------------------------------------------------------------- inputs
def _permuted(values, gen):
    order = torch.randperm(len(values), generator=gen)
    return torch.tensor(values, dtype=torch.int32)[order]


def _table(seq, page, pool, gen, spare=0):
    """Block table of the requests over randomly placed pages (-1 past a
    request's last page), and the pages that nobody holds."""
    have = [-(-s // page) for s in seq]
    width = max(1, max(have) + spare)
    order = torch.randperm(pool, generator=gen).to(torch.int32)
    table = torch.full((len(seq), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:].contiguous()


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


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    page = case["page"]
    if case["op"] == "plan":
        seq = _permuted(_lengths(case), host).tolist()
        new = _permuted(_lengths(case, "new_lo", "new_hi"), host).tolist()
        need = [-(-(s + n) // page) for s, n in zip(seq, new)]
        pool = sum(need) + 16
        spare = max(need) - max(-(-s // page) for s in seq)
        table, free = _table(seq, page, pool, host, spare=max(0, spare))
        return {"op": "plan", "page": page, "tokens": sum(new), "table": table.to(DEV), "free": free.to(DEV),
                "seq": torch.tensor(seq, dtype=torch.int32, device=DEV),
                "new": torch.tensor(new, dtype=torch.int32, device=DEV),
                "start": torch.zeros(1, dtype=torch.int32, device=DEV)}
    dim, heads, heads_kv = case["dim"], case["heads"], case["heads_kv"]
    if case["op"] == "append":
        tokens = case["tokens"]
        pool = -(-tokens // page) + 4
        k_cache, k_scale = _cache(pool, case, gen)
        v_cache, v_scale = _cache(pool, case, gen)
        # keys and values are the last columns of a projection that holds the queries too
        fused = torch.empty((tokens, heads + 2 * heads_kv, dim), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        slots = torch.randperm(pool * page, device=DEV, generator=gen)[:tokens]
        return {"op": "append", "k": fused[:, heads:heads + heads_kv], "v": fused[:, heads + heads_kv:],
                "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale, "slots": slots}
    seq = _permuted(_lengths(case), host).tolist()
    pool = sum(-(-s // page) for s in seq) + 4
    table, _ = _table(seq, page, pool, host)
    k_cache, k_scale = _cache(pool, case, gen)
    v_cache, v_scale = _cache(pool, case, gen)
    q = torch.empty((case["batch"], heads, dim), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    return {"op": "decode", "q": q, "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale,
            "table": table.to(DEV), "seq": torch.tensor(seq, dtype=torch.int32, device=DEV),
            "scale": dim ** -0.5, "window": case["window"]}


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if own:
        import attention_backward_sm_gb300 as fab
        if op == "plan":
            p = fab.kv_plan(state["table"], state["seq"], state["new"], state["free"], state["page"], state["tokens"],
                            free_start=state["start"])
            return {"table": state["table"], "slots": p.slots, "positions": p.positions, "cu_new": p.cu_new,
                    "seq": p.seq_lens, "free_next": p.free_next}
        if op == "append":
            fab.kv_append(state["k"], state["v"], state["k_cache"], state["v_cache"], state["slots"],
                          k_scale=state["k_scale"], v_scale=state["v_scale"])
            return {"k_cache": state["k_cache"], "v_cache": state["v_cache"]}
        o, lse = fab.decode(state["q"], state["k_cache"], state["v_cache"], state["table"], state["seq"],
                            state["scale"], window=state["window"], k_scale=state["k_scale"],
                            v_scale=state["v_scale"])
        return {"o": o, "lse": lse}
    if op == "plan":
        return _plain_plan(**state)
    if op == "append":
        return _plain_append(**state)
    return _plain_decode(**state)


def _plain_plan(op, page, tokens, table, free, seq, new, start):
    have = (seq + page - 1) // page
    after = seq + new
    need = (after + page - 1) // page
    take = need - have
    ends = torch.cumsum(take, 0)
    first = start + ends - take
    at = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (at >= have[:, None]) & (at < need[:, None])
    index = first[:, None] + at - have[:, None]
    pages = free[index.clamp(0, max(free.numel() - 1, 0))] if free.numel() else torch.full_like(table, -1)
    table.copy_(torch.where(fresh, torch.where(index < free.numel(), pages, -1), table))
    cu = torch.zeros(len(seq) + 1, dtype=torch.int64, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    token = torch.arange(tokens, device=table.device)
    b = torch.searchsorted(cu[1:], token, right=True)
    position = seq[b] + token - cu[b]
    held = table[b, position // page].long()
    slots = torch.where(held >= 0, held * page + position % page, -1)
    return {"table": table, "slots": slots, "positions": position.to(torch.int32), "cu_new": cu.to(torch.int32),
            "seq": after, "free_next": (start + ends[-1:]).to(torch.int32)}


def _plain_append(op, k, v, k_cache, v_cache, k_scale, v_scale, slots):
    shape = (-1,) + tuple(k_cache.shape[2:])
    k_cache.view(shape)[slots] = _held(k, k_scale)
    v_cache.view(shape)[slots] = _held(v, v_scale)
    return {"k_cache": k_cache, "v_cache": v_cache}


def _held(x, scale):
    if scale is None:
        return x
    return (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)


def _plain_decode(op, q, k_cache, v_cache, k_scale, v_scale, table, seq, scale, window):
    batch, heads, dim = q.shape
    pool, page, heads_kv, _ = k_cache.shape
    width = table.shape[1] * page
    index = table.clamp(min=0).long()
    k = k_cache[index].view(batch, width, heads_kv, dim).float()
    v = v_cache[index].view(batch, width, heads_kv, dim).float()
    if k_scale is not None:
        k *= k_scale[:, None]
        v *= v_scale[:, None]
    key = torch.arange(width, device=q.device)[None]
    seen = (key < seq[:, None]) & (table >= 0).repeat_interleave(page, 1)
    if window:
        seen &= key >= seq[:, None] - window
    x = torch.matmul(q.view(batch, heads_kv, heads // heads_kv, dim).float(), k.permute(0, 2, 3, 1)) * scale
    x = torch.where(seen[:, None, None], x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, None, None], v, 0.0)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).view(batch, heads)
    return {"o": o.view(batch, heads, dim).to(q.dtype), "lse": lse}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None   # whole numbers
    state = prepare(case, seed)
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            cache, scale = state[name + "_cache"], state[name + "_scale"]
            flat = cache.double().view(-1, *cache.shape[2:])
            new = state[name].double()
            if scale is not None:
                # nearest multiple of the step of the value's power of two (3 fraction bits; 2^-9 near zero), ties to even
                new = new / scale.double()[:, None]
                power = torch.floor(torch.log2(new.abs().clamp(min=2.0 ** -6)))
                step = torch.exp2(power - 3)
                new = (torch.round(new / step) * step).clamp(-448, 448)
            flat.index_copy_(0, state["slots"], new)
            out[name + "_cache"] = flat.view(cache.shape)
        return out
    q = state["q"].double()
    batch, heads, dim = q.shape
    heads_kv, page, window = case["heads_kv"], case["page"], case["window"]
    table, seq = state["table"].long(), state["seq"].tolist()
    o = torch.zeros_like(q)
    lse = torch.full((batch, heads), float("-inf"), dtype=torch.float64, device=DEV)
    for b, n in enumerate(seq):
        at = torch.arange(max(0, n - window) if window else 0, n, device=DEV)
        if not len(at):
            continue
        pages = table[b, at // page]
        k = state["k_cache"][pages, at % page].double().transpose(0, 1)
        v = state["v_cache"][pages, at % page].double().transpose(0, 1)
        if state["k_scale"] is not None:
            k = k * state["k_scale"].double()[:, None, None]
            v = v * state["v_scale"].double()[:, None, None]
        x = case["dim"] ** -0.5 * torch.bmm(q[b].view(heads_kv, -1, dim), k.transpose(1, 2))
        lse[b] = torch.logsumexp(x, -1).view(-1)
        o[b] = torch.bmm(torch.softmax(x, -1), v).view(heads, dim)
    return {"o": o, "lse": lse}
