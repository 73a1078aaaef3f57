"""What the paged 4-bit KV cache operators are measured on.

Three operators of the serving path, which belong together:

* plan   -- `kv_plan`: block tables, slots and positions of a step's new tokens,
            built on the GPU from the requests' lengths;
* append -- `kv_append`: the new K and V rows quantized (NVFP4 or MXFP4) into
            their slots of the paged cache;
* attend -- `kv_attention`: causal attention of the step's queries over the
            cache, from one token a request (decode) to long prompts (prefill).

A case is a dict of plain values; lengths follow from the case alone (spread
evenly over their range, dealt to the requests by the seed), so `work` is exact.
Where `own` is false `run` computes the operators from elementary torch
operations in 32 bits; where it is true it makes the framework's calls.
"""
import math
import random

import torch

own = False

# ------------------------------------------------------------------- cases


def _plan(name, batch, page, cached, new, pad):
    return {"name": name, "op": "plan", "batch": batch, "page": page, "cached_lo": cached[0], "cached_hi": cached[1],
            "new_lo": new[0], "new_hi": new[1], "pad": pad}


def _append(name, mode, batch, kv_heads, q_heads, dim, page, cached, new, global_scale):
    return {"name": name, "op": "append", "mode": mode, "batch": batch, "kv_heads": kv_heads, "q_heads": q_heads,
            "dim": dim, "page": page, "cached_lo": cached[0], "cached_hi": cached[1], "new_lo": new[0],
            "new_hi": new[1], "global_scale": global_scale}


def _attend(name, mode, batch, q_heads, kv_heads, dim, page, cached, new, window, global_scale):
    return {"name": name, "op": "attend", "mode": mode, "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "cached_lo": cached[0], "cached_hi": cached[1], "new_lo": new[0],
            "new_hi": new[1], "window": window, "global_scale": global_scale}


def listed():
    return [
        # one decode step of a busy server: every request adds a token, some of them cross into a new page
        _plan("plan, 64 requests decode", 64, 64, (1, 8191), (1, 1), 0),
        # a step that mixes idle requests, decodes and prompt chunks, padded to a fixed token count as a captured graph needs
        _plan("plan, 1000 requests mixed", 1000, 16, (0, 4096), (0, 129), 500),
        # the smallest write: one new token of one request, all 40 heads of the hidden-5120 stack
        _append("append, 1 token", "nvfp4", 1, 40, 40, 128, 64, (300, 300), (1, 1), True),
        # prompts of several requests written in one step, grouped heads, small pages
        _append("append, prompts of 7 requests", "mxfp4", 7, 8, 64, 128, 16, (0, 333), (1, 4999), False),
        # interactive decode: a single request, a short odd context, one kv head per query head
        _attend("decode, 1 x 997", "nvfp4", 1, 40, 40, 128, 64, (996, 996), (1, 1), 0, True),
        # ordinary decode batch: grouped heads, ragged contexts
        _attend("decode, 32 x 1..8k", "nvfp4", 32, 64, 8, 128, 64, (0, 8191), (1, 1), 0, True),
        # one very long context: the work has to be split along it
        _attend("decode, 1 x 131k", "nvfp4", 1, 64, 8, 128, 128, (131076, 131076), (1, 1), 0, False),
        # the largest decode batch: gigabytes of cache read in a step
        _attend("decode, 96 x 4k..20k", "mxfp4", 96, 40, 8, 128, 32, (4000, 20000), (1, 1), 0, False),
        # head size 64 with a sliding window and small pages, and requests that have only just begun
        _attend("decode, 24 x window 128", "mxfp4", 24, 64, 8, 64, 16, (0, 6000), (1, 1), 128, False),
        # a few tokens a request: checking drafted tokens
        _attend("verify, 16 x 4 tokens", "nvfp4", 16, 64, 8, 128, 64, (100, 8003), (4, 4), 0, True),
        # a whole prompt from an empty cache at the hidden-5120 stack's heads
        _attend("prefill, 1 x 4096", "nvfp4", 1, 40, 40, 128, 64, (0, 0), (4096, 4096), 0, True),
        # chunks of several prompts over what is already cached, head size 64
        _attend("prefill, 4 chunks over 0..16k", "mxfp4", 4, 64, 8, 64, 32, (0, 16001), (100, 1023), 0, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    mode = rng.choice(["nvfp4", "mxfp4"])
    gs = mode == "nvfp4" and rng.random() < 0.6
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        lo, new = _log(rng, 1, 4000) - 1, _log(rng, 1, 128)
        c = _plan("", _log(rng, 1, 1000), page, (lo, lo + _log(rng, 1, 4000)), (rng.randint(0, 1), new),
                  rng.choice([0, _log(rng, 1, 1000)]))
    else:
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 5, 8, 8, 40])
        group = rng.choice([1, 2, 5, 8, 16]) if kv < 40 else 1
        if op == "append":
            batch, lo, new = _log(rng, 1, 32), _log(rng, 1, 500) - 1, _log(rng, 1, 16384)
            new = max(1, min(new, 17000 * 8 // (batch * kv)))
            c = _append("", mode, batch, kv, kv * group, dim, page, (lo, lo + _log(rng, 1, 400)),
                        (max(1, new // 3), new), gs)
        elif rng.random() < 0.6:  # decode
            batch = _log(rng, 1, 128)
            hi = min(_log(rng, 1, 131072), 9_000_000 // (batch * kv))
            c = _attend("", mode, batch, kv * group, kv, dim, page, (rng.randint(0, hi), hi), (1, 1),
                        rng.choice([0, 0, _log(rng, 1, 4096)]), gs)
        else:  # several tokens a request
            batch, hi = _log(rng, 1, 16), _log(rng, 2, 4096)
            cached = _log(rng, 1, 16000) - 1
            # at most about the multiplications of the largest prefill listed
            room = 250_000_000 // (batch * kv * group)
            while hi * (cached + hi) > room and hi * (cached + hi) > 64:
                hi, cached = max(2, hi * 2 // 3), cached * 2 // 3
            c = _attend("", mode, batch, kv * group, kv, dim, page, (rng.randint(0, cached), cached),
                        (max(1, hi // 2), hi), rng.choice([0, 0, 0, _log(rng, 1, 4096)]), gs)
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [(lo + hi) // 2]


def _lengths(case, seed=None):
    """(cached, new) lengths of the requests; a seed deals the pairs out in its own order."""
    n = case["batch"]
    cached = _spread(case["cached_lo"], case["cached_hi"], n)
    new = _spread(case["new_lo"], case["new_hi"], n)
    new = new[1::2] + new[0::2]  # long contexts do not always get the long chunks
    pairs = list(zip(cached, new))
    if seed is not None:
        random.Random(seed).shuffle(pairs)
    return [p[0] for p in pairs], [p[1] for p in pairs]


def _pages(length, page):
    return -(-length // page)


# ------------------------------------------------- the 4-bit formats, plain

_GROUP = {"nvfp4": 16, "mxfp4": 32}
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _quantize(x, mode, gs):
    """The framework's rule in 32 bits: x [..., D] float32 -> (codes int32 [..., D/8], scales uint8 [..., D/group])."""
    g = _GROUP[mode]
    xg = x.reshape(*x.shape[:-1], -1, g)
    b = xg.abs().amax(-1)
    if mode == "nvfp4":
        gs = torch.ones((), device=x.device) if gs is None else gs
        s = torch.where(b == 0, torch.zeros_like(b), b / (6.0 * gs)).clamp(max=448.0)
        s8 = s.to(torch.float8_e4m3fn)
        d = s8.float() * gs
        mul = torch.where(d == 0, torch.zeros_like(d), 1.0 / d)
        scales = s8.view(torch.uint8)
    else:
        e = torch.frexp(b).exponent - 1  # floor(log2 b)
        se = torch.where(b == 0, torch.full_like(e, -127), (e - 2).clamp(-127, 127))
        mul = torch.ldexp(torch.ones_like(b), -se)
        scales = (se + 127).to(torch.uint8)
    v = xg * mul[..., None]
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = (code + 8 * torch.signbit(v).int()).reshape(*x.shape[:-1], -1, 8)
    shift = torch.arange(0, 32, 4, device=x.device, dtype=torch.int64)
    words = (code.long() << shift).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), scales


def _scale_values(scales, mode):
    if mode == "nvfp4":
        return scales.view(torch.float8_e4m3fn).float()
    return torch.ldexp(torch.ones((), device=scales.device), scales.int() - 127)


def _values(codes, scales, mode, gs):
    """codes int32 [..., D/8], scales uint8 [..., D/group] -> the values they stand for, float32 [..., D]."""
    table = torch.tensor(_E2M1, device=codes.device)
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)  # byte -> (low code, high code)
    v = pairs[codes.contiguous().view(torch.uint8).int()].flatten(-2)
    g = _GROUP[mode]
    v = (v.view(*scales.shape, g) * _scale_values(scales, mode)[..., None]).flatten(-2)
    return v if gs is None else v * gs


# ----------------------------------------------------------------- inputs


def _rows(n, heads, dim, gen, std, dev):
    """Key or value rows as a model makes them: normal, with a few channels that are larger throughout."""
    x = torch.randn((n, heads, dim), generator=gen, device=dev) * std
    big = torch.rand((heads, dim), generator=gen, device=dev) < 0.03
    return x * torch.where(big, 4.0, 1.0)


def _global_scale(x):
    return (x.abs().amax() / 2688.0).float()


def _fill(case, seed, pages, dev, gen):
    """A paged cache whose slots all hold quantized rows (freed pages hold old ones)."""
    mode, kv, dim, page = case["mode"], case["kv_heads"], case["dim"], case["page"]
    state = {}
    pool = 4096
    for which, std in (("k", 1.0), ("v", 0.7)):
        x = _rows(pool, kv, dim, gen, std, dev).to(torch.bfloat16).float()
        gs = _global_scale(x) if case["global_scale"] else None
        codes, scales = _quantize(x, mode, gs)
        pick = torch.randint(0, pool, (pages * page,), generator=gen, device=dev)
        for name, t in (("codes", codes), ("scales", scales)):
            full = torch.empty((pages, kv, page, t.shape[-1]), dtype=t.dtype, device=dev)
            for h in range(kv):
                full[:, h] = t[:, h][pick].view(pages, page, -1)
            state[which + "_" + name] = full
        state["gs_" + which] = gs
    return state


def _table(total, page, pages, max_pages, seed, dev):
    """Block table of requests of `total` tokens each: distinct pages in no order; unused entries 0."""
    order = list(range(pages))
    random.Random(seed + 1).shuffle(order)
    rows, at = [], 0
    for n in total:
        k = _pages(n, page)
        rows.append(order[at:at + k] + [0] * (max_pages - k))
        at += k
    return torch.tensor(rows, dtype=torch.int32, device=dev), order[at:]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    cached, new = _lengths(case, seed)
    total = [a + b for a, b in zip(cached, new)]
    page = case["page"]
    max_pages = max(1, max(_pages(n, page) for n in total))
    tokens = sum(new)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    state = {"case": case, "cached_lens": ints(cached), "new_lens": ints(new), "tokens": tokens}
    if case["op"] == "plan":
        pages = sum(_pages(n, page) for n in total) + 64
        state["block_table"], free = _table(cached, page, pages, max_pages, seed, dev)
        state["free_pages"] = ints(free)
        state["tokens"] = tokens + case["pad"]
        return state
    spare = 2
    pages = sum(_pages(n, page) for n in total) + spare
    state.update(_fill(case, seed, pages, dev, gen))
    state["block_table"], _ = _table(total, page, pages, max_pages, seed, dev)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    state["query_start"], state["total_lens"] = ints(starts), ints(total)
    state["max_query_len"], state["max_total_len"] = max(new), max(total)
    heads, kv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    # q, k and v of the step's tokens as the fused projection leaves them: one row of all heads a token
    qkv = torch.empty((tokens, heads + 2 * kv, dim), dtype=torch.bfloat16, device=dev)
    if case["op"] == "append":
        qkv[:, heads:heads + kv] = _rows(tokens, kv, dim, gen, 1.0, dev).to(torch.bfloat16)
        qkv[:, heads + kv:] = _rows(tokens, kv, dim, gen, 0.7, dev).to(torch.bfloat16)
        state["k"], state["v"] = qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        req = torch.repeat_interleave(torch.arange(len(new), device=dev), state["new_lens"].long())
        pos = state["cached_lens"][req] + torch.arange(tokens, device=dev) - state["query_start"][req]
        state["slot_map"] = state["block_table"][req, pos // page].long() * page + pos % page
    else:
        qkv[:, :heads] = (1.5 * torch.randn((tokens, heads, dim), generator=gen, device=dev)).to(torch.bfloat16)
        state["q"] = qkv[:, :heads]
    return state


# -------------------------------------------------------------- plain forms


def _plain_plan(s):
    page, table = s["case"]["page"], s["block_table"]
    cached, new, free = s["cached_lens"].long(), s["new_lens"].long(), s["free_pages"]
    total = cached + new
    old, need = (cached + page - 1) // page, (total + page - 1) // page
    take = need - old
    first = torch.cumsum(take, 0) - take
    starts = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= old[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - old[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[at], table)
    t = torch.arange(s["tokens"], device=table.device)
    real = t < starts[-1]
    req = torch.searchsorted(starts[1:], t, right=True).clamp(max=cached.numel() - 1)
    pos = (cached[req] + t - starts[req]).clamp(min=0)
    slot = table[req, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    return {"block_table": table, "total_lens": total.int(), "query_start": starts.int(),
            "slot_map": torch.where(real, slot, -1), "positions": torch.where(real, pos, -1).int(),
            "pages_taken": take.sum().int()}


def _plain_append(s):
    mode, page = s["case"]["mode"], s["case"]["page"]
    p, o = s["slot_map"] // page, s["slot_map"] % page
    out = {}
    for which in ("k", "v"):
        codes, scales = _quantize(s[which].float(), mode, s["gs_" + which])
        s[which + "_codes"][p, :, o] = codes
        s[which + "_scales"][p, :, o] = scales
        out[which] = _values(s[which + "_codes"], s[which + "_scales"], mode, s["gs_" + which]).to(torch.bfloat16)
    return out


def _plain_attend(s):
    c = s["case"]
    mode, page, kv, dim = c["mode"], c["page"], c["kv_heads"], c["dim"]
    group = c["q_heads"] // kv
    starts, total = s["query_start"].long(), s["total_lens"].long()
    batch, rows, length = total.numel(), s["max_query_len"], s["max_total_len"]
    dev = total.device
    # the requests' queries side by side, padded to the longest: [batch, kv head, group * rows, dim]
    i = torch.arange(rows, device=dev)
    t = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][t].float().view(batch, rows, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, group * rows, dim)
    # and their keys: [batch, kv head, length, dim]
    j = torch.arange(length, device=dev)
    pages, slots = s["block_table"][:, j // page].long(), (j % page).expand(batch, -1)

    def gathered(which):
        v = _values(s[which + "_codes"][pages, :, slots], s[which + "_scales"][pages, :, slots], mode, s["gs_" + which])
        return v.transpose(1, 2)

    score = q @ gathered("k").transpose(2, 3) * dim ** -0.5
    pos = total[:, None] - (starts[1:] - starts[:-1])[:, None] + i  # [batch, rows]
    seen = (j <= pos[..., None]) & (j < total[:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    score = score.view(batch, kv, group, rows, length).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    sums = p.sum(-1, keepdim=True)
    p = p.view(batch, kv, group * rows, length)
    o = (p @ gathered("v")).view(batch, kv, group, rows, dim)
    o = torch.where(sums > 0, o / sums, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, rows, kv * group, dim)
    t = torch.arange(s["q"].shape[0], device=dev)
    req = torch.searchsorted(starts[1:], t, right=True)
    return o[req, t - starts[req]].to(torch.bfloat16)


# --------------------------------------------------------------------- run


def _cache(s):
    from block_scaled_fp4_fp_gb300 import binding as B
    if "cache" not in s:
        mode = B.MODE_NVFP4 if s["case"]["mode"] == "nvfp4" else B.MODE_MXFP4
        s["cache"] = B.kv_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], mode, s["gs_k"], s["gs_v"])
    return s["cache"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[op](s)
    from block_scaled_fp4_fp_gb300 import binding as B
    if op == "plan":
        plan = B.kv_plan(s["cached_lens"], s["new_lens"], s["free_pages"], s["block_table"], s["case"]["page"],
                         s["tokens"])
        return {"block_table": s["block_table"], "total_lens": plan.total_lens, "query_start": plan.query_start,
                "slot_map": plan.slot_map, "positions": plan.positions, "pages_taken": plan.pages_taken}
    cache = _cache(s)
    if op == "append":
        B.kv_append(cache, s["k"], s["v"], s["slot_map"])
        out = {}
        for which in ("k", "v"):  # the cache is four matrices of the framework's formats: its own call reads them
            codes, scales = s[which + "_codes"], s[which + "_scales"]
            out[which] = B.fp4_dequantize(codes.view(-1, codes.shape[-1]), scales.view(-1, scales.shape[-1]),
                                          mode=cache.mode, global_scale=s["gs_" + which])
            out[which] = out[which].view(*codes.shape[:-1], -1)
        return out
    if "ws" not in s:
        s["ws"] = B.kv_attention_workspace(cache, s["total_lens"].numel(), s["q"].shape[1], s["max_query_len"])
    return B.kv_attention(cache, s["q"], s["query_start"], s["total_lens"], s["block_table"], s["ws"],
                          max_query_len=s["max_query_len"], window=s["case"]["window"])


# ---------------------------------------------------------- work and exact


def _seen(case):
    """(sum over requests of keys any query sees, sum over query rows of keys seen), per kv head / query head."""
    keys = pairs = 0
    w = case["window"]
    for c, n in zip(*_lengths(case)):
        if n == 0:
            continue
        if w:
            first = max(0, c + 1 - w)
            keys += c + n - first
            full = max(0, min(n, w - c))  # rows whose window still holds every key before them
            pairs += full * c + full * (full + 1) // 2 + (n - full) * w
        else:
            keys += c + n
            pairs += n * c + n * (n + 1) // 2
    return keys, pairs


def work(case):
    cached, new = _lengths(case)
    tokens, page = sum(new), case["page"]
    if case["op"] == "plan":
        total_pages = sum(_pages(a + b, page) for a, b in zip(cached, new))
        taken = total_pages - sum(_pages(a, page) for a in cached)
        read = 8 * case["batch"] + 4 * taken + 4 * case["batch"]
        return {"bytes": read + 4 * taken + 8 * case["batch"] + 12 * (tokens + case["pad"]), "flops": 0}
    kv, dim = case["kv_heads"], case["dim"]
    row = dim / 2 + dim / _GROUP[case["mode"]]  # bytes of one cached row
    if case["op"] == "append":
        pages = sum(_pages(a + b, page) for a, b in zip(cached, new)) + 2
        rows = pages * page
        # new rows read and written; the whole cache read once and its values written
        return {"bytes": 2 * kv * (tokens * (2 * dim + row) + rows * (row + 2 * dim)) + 8 * tokens, "flops": 0}
    keys, pairs = _seen(case)
    return {"bytes": 2 * kv * keys * row + 4 * tokens * case["q_heads"] * dim + 4 * _pages(keys, page),
            "flops": 4 * pairs * case["q_heads"] * dim}


def _exact_values(codes, scales, mode, gs):
    """Values of stored codes in 64 bits, from the formats' bit fields."""
    word = codes.long() & 0xFFFFFFFF
    nib = torch.stack([(word >> (4 * k)) & 15 for k in range(8)], -1).flatten(-2)
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    v = torch.where(nib >= 8, -mag, mag)
    b = scales.long()
    if mode == "nvfp4":
        se, sm = (b >> 3) & 15, (b & 7).double()
        sc = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8) * torch.pow(2.0, (se - 7).double()))
    else:
        sc = torch.pow(2.0, (b - 127).double())
    v = v * sc.repeat_interleave(v.shape[-1] // sc.shape[-1], -1)
    return v if gs is None else v * gs.double()


def _nearest(x, grid):
    """Nearest of the sorted grid's values to each |x| (ties to the even place), with x's sign."""
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
    lo = hi - 1
    below, above = a - grid[lo], grid[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(torch.signbit(x), -1.0, 1.0) * grid[torch.where(up, hi, lo)]


def _exact_append(s):
    case = s["case"]
    mode, page, g = case["mode"], case["page"], _GROUP[case["mode"]]
    out = {}
    dev = s["slot_map"].device
    e2m1 = torch.tensor(_E2M1[:8], dtype=torch.float64, device=dev)
    e4m3 = torch.tensor(sorted([m * 2.0 ** -9 for m in range(8)]
                               + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])[:-1],
                        dtype=torch.float64, device=dev)
    for which in ("k", "v"):
        x = s[which].double()
        x = x.reshape(*x.shape[:2], -1, g)
        gs = s["gs_" + which]
        top = x.abs().amax(-1, keepdim=True)
        if mode == "nvfp4":
            one = 1.0 if gs is None else gs.double()
            step = _nearest(top / (6 * one), e4m3) * one
        else:
            step = torch.where(top > 0, torch.pow(2.0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 2), 2.0 ** -127)
        v = torch.where(step > 0, _nearest(x / step.clamp(min=1e-300), e2m1) * step, 0.0).flatten(-2)
        whole = _exact_values(s[which + "_codes"], s[which + "_scales"], mode, gs)
        whole[s["slot_map"] // page, :, s["slot_map"] % page] = v
        out[which] = whole
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    kv, dim, page, w = case["kv_heads"], case["dim"], case["page"], case["window"]
    group = case["q_heads"] // kv
    keys, pairs = _seen(case)
    if pairs * case["q_heads"] * dim > 2e12 or keys * kv * dim > 4e9:
        return None
    out = torch.zeros((s["q"].shape[0], case["q_heads"], dim), dtype=torch.float64, device=s["q"].device)
    starts, total = s["query_start"].tolist(), s["total_lens"].tolist()
    for b, n in enumerate(total):
        a, z = starts[b], starts[b + 1]
        if z == a:
            continue
        first = max(0, n - (z - a) + 1 - w) if w else 0
        where = torch.arange(first, n, device=out.device)
        pages, slots = s["block_table"][b, where // page].long(), where % page
        pos = n - (z - a) + torch.arange(z - a, device=out.device)
        hidden = where > pos[:, None]
        if w:
            hidden |= where <= pos[:, None] - w
        for h in range(kv):
            k, v = (_exact_values(s[x + "_codes"][pages, h, slots], s[x + "_scales"][pages, h, slots], case["mode"],
                                  s["gs_" + x]) for x in ("k", "v"))
            q = s["q"][a:z, h * group:(h + 1) * group].double().transpose(0, 1)
            score = (q @ k.T) / math.sqrt(dim)
            out[a:z, h * group:(h + 1) * group] = (torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v).transpose(0, 1)
    return out
