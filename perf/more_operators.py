"""What the operators around a decoder layer's 4-bit products are measured on.

Four groups, which a layer calls one after the other:

* norm    -- `rms_norm`: the residual added, the root-mean-square norm, out in bf16 or quantized for the next product;
* rope    -- `rope`: rotary positions on a [tokens, heads, head_dim] view, or their gradient;
* append  -- `kv_append_rope`: new K rotated and quantized with V into the paged 4-bit cache, q rotated beside them;
* sort    -- `moe_sort`: the routed rows in order of their experts, as `gather_qmm` wants them;
* combine -- `moe_combine` and `moe_combine_backward`: the experts' rows back to their tokens, weighted, and the gradients.

A case is a dict of plain values.  Where `own` is false `run` computes the
operators from elementary torch operations; where it is true it makes the
framework's calls.  32 bits throughout, but for a row's mean square and the
angles, which are formed in 64: one unit in the last place of either moves an
element next to a rounding border of the 4-bit formats by a whole step.
"""
import math
import random

import torch

own = False

# ------------------------------------------------------------------- cases


def _norm(name, rows, cols, residual, out, tiled, global_scale, pad):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "residual": residual, "out": out, "tiled": tiled,
            "global_scale": global_scale, "pad": pad}


def _rope(name, tokens, heads, dim, rotary, interleaved, far, scaling, backward):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "far": far, "scaling": scaling, "backward": backward}


def _append(name, mode, batch, q_heads, kv_heads, dim, page, cached, new, rotary, interleaved, scaling, pad, global_scale):
    return {"name": name, "op": "append", "mode": mode, "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "cached_lo": cached[0], "cached_hi": cached[1], "new_lo": new[0], "new_hi": new[1],
            "rotary": rotary, "interleaved": interleaved, "scaling": scaling, "pad": pad, "global_scale": global_scale}


def _sort(name, tokens, k, experts, pad):
    return {"name": name, "op": "sort", "tokens": tokens, "k": k, "experts": experts, "pad": pad}


def _combine(name, tokens, k, experts, cols, weights, residual, pad, backward):
    return {"name": name, "op": "combine", "tokens": tokens, "k": k, "experts": experts, "cols": cols, "weights": weights,
            "residual": residual, "pad": pad, "backward": backward}


def listed():
    return [
        # one token of a request on its own, in front of the 4-bit GEMV
        _norm("norm, 1 x 5120", 1, 5120, True, "bf16", False, False, 0),
        # a prompt in front of the 4-bit GEMM, which reads its activations quantized with tiled scales
        _norm("norm, 4096 x 5120 to nvfp4", 4096, 5120, True, "nvfp4", True, True, 0),
        # an odd number of rows of another width, without a residual
        _norm("norm, 8001 x 2880 to mxfp4", 8001, 2880, False, "mxfp4", False, False, 0),
        # the query heads of a prompt, whole heads in halves, far into a long context
        _rope("rope, 4096 x 40 of 128", 4096, 40, 128, 128, False, 131072, "ramp", False),
        # the gradient of an interleaved rotation of half of each head
        _rope("rope gradient, 1001 x 64 of 64", 1001, 64, 64, 32, True, 8192, "none", True),
        # a serving step: a token of each of 64 requests, padded as a captured graph needs
        _append("append, 64 tokens", "nvfp4", 64, 64, 8, 128, 16, (0, 31), (1, 1), 128, False, "wavelength", 16, True),
        # prompts of several requests
        _append("append, prompts of 7 requests", "mxfp4", 7, 32, 8, 128, 64, (0, 333), (1, 4999), 128, False, "linear", 0, False),
        # a serving step's routing
        _sort("sort, 96 x 4 of 32", 96, 4, 32, 0),
        # a long prompt's over many experts
        _sort("sort, 16384 x 8 of 256", 16384, 8, 256, 300),
        # a serving step's rows back to its tokens, on top of the residual
        _combine("combine, 96 x 4 of 5120", 96, 4, 32, 5120, True, True, 0, False),
        # a prompt's
        _combine("combine, 2048 x 4 of 2880", 2048, 4, 32, 2880, True, False, 0, False),
        # and its gradients
        _combine("combine gradient, 2048 x 4", 2048, 4, 32, 2880, True, False, 50, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rope", "append", "append", "sort", "combine", "combine"])
    if op == "norm":
        cols = 32 * _log(rng, 2, 544)
        rows = min(_log(rng, 1, 100000), 21_000_000 // cols)
        out = rng.choice(["bf16", "nvfp4", "mxfp4"])
        c = _norm("", rows, cols, rng.random() < 0.6, out, out != "bf16" and rng.random() < 0.5,
                  out == "nvfp4" and rng.random() < 0.6, rng.choice([0, 0, 8 * rng.randint(1, 40)]))
    elif op == "rope":
        dim = rng.choice([64, 96, 128, 128, 256])
        heads = rng.choice([1, 2, 5, 8, 16, 40, 64])
        tokens = min(_log(rng, 1, 16384), 20_000_000 // (heads * dim))
        c = _rope("", tokens, heads, dim, rng.choice([dim, dim, dim // 2, dim // 4]), rng.random() < 0.4,
                  _log(rng, 20000, 131072), rng.choice(["none", "linear", "base", "wavelength", "ramp"]), rng.random() < 0.3)
    elif op == "append":
        dim = rng.choice([64, 96, 128, 128, 256])
        kv = rng.choice([1, 2, 5, 8, 8, 40])
        heads = kv * (rng.choice([1, 2, 4, 5, 8]) if kv < 40 else 1)
        batch = min(_log(rng, 1, 128), 20_000_000 // (kv * dim * 400))
        new = 1 if rng.random() < 0.4 else _log(rng, 2, 8000)
        new = max(1, min(new, 40_000_000 // (batch * (heads + 2 * kv) * dim)))
        lo = rng.randint(0, 100)
        mode = rng.choice(["nvfp4", "mxfp4"])
        c = _append("", mode, batch, heads, kv, dim, rng.choice([16, 32, 64, 128]), (lo, lo + rng.randint(0, 100)),
                    (max(1, new // 3), new), rng.choice([dim, dim, dim // 2, dim // 4]), rng.random() < 0.4,
                    rng.choice(["none", "linear", "base", "wavelength", "ramp"]), rng.choice([0, 0, rng.randint(1, 40)]),
                    mode == "nvfp4" and rng.random() < 0.6)
    else:
        experts = rng.choice([4, 8, 32, 60, 128, 256])
        k = rng.choice([x for x in (1, 2, 3, 4, 6, 8) if x <= experts])
        if op == "sort":
            tokens = _log(rng, 1, 16384)
            c = _sort("", tokens, k, experts, rng.choice([0, rng.randint(0, tokens)]))
        else:
            cols = 8 * _log(rng, 16, 900)
            tokens = min(_log(rng, 1, 8192), 24_000_000 // (k * cols))
            back = rng.random() < 0.5
            c = _combine("", tokens, k, experts, cols, rng.random() < 0.8, not back and rng.random() < 0.5,
                         rng.choice([0, rng.randint(0, tokens // 2)]), back)
    del c["name"]
    return c


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


def _values(codes, scales, mode, gs):
    """codes int32 [..., D/8], scales uint8 [..., D/group] -> the values they stand for, bf16 [..., D]."""
    table = torch.tensor(_E2M1, device=codes.device)
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)  # byte -> (low code, high code)
    v = pairs[codes.contiguous().view(torch.uint8).int()].flatten(-2)
    s = (scales.view(torch.float8_e4m3fn).float() if mode == "nvfp4"
         else torch.ldexp(torch.ones((), device=scales.device), scales.int() - 127))
    v = (v.view(*scales.shape, _GROUP[mode]) * s[..., None]).flatten(-2)
    return (v if gs is None else v * gs).to(torch.bfloat16)


# ------------------------------------------------------- rotary frequencies

_BASE = 10000.0
#: scaling -> (factor, original positions, low, high) as the framework's frequencies take them
_SCALING = {"none": (1.0, 1, 1.0, 1.0), "linear": (4.0, 1, 1.0, 1.0), "base": (8.0, 1, 1.0, 1.0),
            "wavelength": (8.0, 8192, 1.0, 4.0), "ramp": (16.0, 4096, 1.0, 32.0)}


def _frequencies(rotary, scaling):
    """(radians a position for each pair, what cos and sin are multiplied by), in 64 bits."""
    factor, original, low, high = _SCALING[scaling]
    f = [_BASE ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    if scaling == "linear":  # positions as if the context were shorter
        return [x / factor for x in f], 1.0
    if scaling == "base":  # a larger base: the slowest pair is stretched by the factor, the fastest not at all
        base = _BASE * factor ** (rotary / (rotary - 2.0)) if rotary > 2 else _BASE
        return [base ** (-2.0 * i / rotary) for i in range(rotary // 2)], 1.0
    if scaling == "wavelength":  # long waves stretched, short ones kept, a blend between
        out = []
        for x in f:
            turns = original * x / (2 * math.pi)  # of the pair over the original context
            s = min(1.0, max(0.0, (turns - low) / (high - low)))
            out.append((1 - s) * x / factor + s * x)
        return out, 1.0
    if scaling == "ramp":  # the same over the pairs' numbers, and scores sharpened
        at = lambda turns: rotary * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(_BASE))  # noqa: E731
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rotary - 1)
        out = []
        for i, x in enumerate(f):
            s = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            out.append(x / factor * s + x * (1 - s))
        return out, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _cos_sin(positions, rotary, scaling):
    """cos and sin in 64 bits, [..., rotary/2] each."""
    f, scale = _frequencies(rotary, scaling)
    a = positions.double()[..., None] * torch.tensor(f, dtype=torch.float64, device=positions.device)
    return torch.cos(a) * scale, torch.sin(a) * scale


def _rotated(x, cos, sin, rotary, interleaved):
    """x [tokens, heads, dim], cos and sin [tokens, rotary/2]."""
    cos, sin = cos[:, None], sin[:, None]
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rotary // 2], r[..., rotary // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, x[..., rotary:]], -1)


# ----------------------------------------------------------------- inputs


def _pages(length, page):
    return -(-length // page)


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [(lo + hi) // 2]


def _lengths(case, seed=None):
    """(cached, new) lengths of the requests; a seed deals the pairs out in its own order."""
    n = case["batch"]
    pairs = list(zip(_spread(case["cached_lo"], case["cached_hi"], n), _spread(case["new_lo"], case["new_hi"], n)))
    if seed is not None:
        random.Random(seed).shuffle(pairs)
    return [p[0] for p in pairs], [p[1] for p in pairs]


def _cache_pages(case):
    return sum(_pages(a + b, case["page"]) for a, b in zip(*_lengths(case))) + 1


def _activations(shape, gen, dev):
    """Rows as a model's residual stream has them: normal, with a few channels that are larger throughout."""
    x = torch.randn(shape, generator=gen, device=dev)
    return x * torch.where(torch.rand(shape[-1], generator=gen, device=dev) < 0.02, 8.0, 1.0)


def _routing(case, gen, dev):
    """Distinct experts of each token, some of them popular; the padding tokens at the end have none (-1)."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    score = torch.randn((t, e), generator=gen, device=dev) + torch.randn(e, generator=gen, device=dev)
    top = score.topk(k)
    ids = top.indices.int()
    if case["pad"]:
        ids[t - case["pad"]:] = -1
    return ids, torch.softmax(top.values, -1)


def _prepare_append(case, seed, gen, dev, state):
    mode, kv, heads, dim, page = case["mode"], case["kv_heads"], case["q_heads"], case["dim"], case["page"]
    cached, new = _lengths(case, seed)
    pages, n, pad = _cache_pages(case), sum(new), case["pad"]
    order = list(range(pages))
    random.Random(seed + 1).shuffle(order)
    slots, positions, at = [], [], 0
    for c, m in zip(cached, new):
        mine = torch.tensor(order[at:at + _pages(c + m, page)], dtype=torch.int64)
        at += len(mine)
        pos = torch.arange(c, c + m)
        slots.append(mine[pos // page] * page + pos % page)
        positions.append(pos)
    gone = torch.full((pad,), -1, dtype=torch.int64)
    state["slot_map"] = torch.cat(slots + [gone]).to(dev)
    state["positions"] = torch.cat(positions + [gone]).int().to(dev)
    state["real"] = n
    # q, k and v as the fused projection leaves them: one row of all heads a token
    qkv = torch.randn((n + pad, heads + 2 * kv, dim), generator=gen, device=dev)
    qkv = (qkv * torch.where(torch.rand((heads + 2 * kv, dim), generator=gen, device=dev) < 0.03, 4.0, 1.0)).bfloat16()
    state["q"], state["k"], state["v"] = qkv.split([heads, kv, kv], 1)
    state["q_out"] = torch.zeros((n + pad, heads, dim), dtype=torch.bfloat16, device=dev)
    for which in ("k", "v"):
        state[which + "_codes"] = torch.randint(-2 ** 31, 2 ** 31, (pages, kv, page, dim // 8), generator=gen, device=dev).int()
        lo, hi = (40, 90) if mode == "nvfp4" else (120, 128)
        state[which + "_scales"] = torch.randint(lo, hi, (pages, kv, page, dim // _GROUP[mode]), generator=gen,
                                                 device=dev).to(torch.uint8)
        # calibrated once for the cache's life: of no simple ratio to this step's values
        state["gs_" + which] = torch.tensor(0.00719431, device=dev) if case["global_scale"] else None
    state["far"] = 1 + max(c + m for c, m in zip(cached, new))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        state["x"] = _activations((rows, cols + case["pad"]), gen, dev).bfloat16()[:, :cols]
        state["residual"] = (3 * _activations((rows, cols), gen, dev)).bfloat16() if case["residual"] else None
        state["weight"] = (1 + 0.2 * torch.randn(cols, generator=gen, device=dev)).bfloat16()
        state["eps"] = 1e-6
        # a calibrated scale of the normed activations
        state["gs"] = torch.tensor(0.00743119, device=dev) if case["global_scale"] else None
    elif case["op"] == "rope":
        t = case["tokens"]
        qkv = torch.randn((t, case["heads"] + 2, case["dim"]), generator=gen, device=dev).bfloat16()
        state["x"] = qkv[:, :case["heads"]]
        first = random.Random(seed).randint(0, case["far"] - t)
        state["positions"] = torch.arange(first, first + t, dtype=torch.int32, device=dev)
        state["far"] = case["far"]
    elif case["op"] == "append":
        _prepare_append(case, seed, gen, dev, state)
    else:
        state["ids"], weights = _routing(case, gen, dev)
        if case["op"] == "combine":
            t, k, n = case["tokens"], case["k"], case["cols"]
            plan = _plain_sort(state)
            state["slot"], state["offsets"] = plan["slot"], plan["offsets"]
            state["weights"] = weights if case["weights"] else None
            state["y"] = torch.randn((t * k, n), generator=gen, device=dev).bfloat16()
            state["residual"] = (3 * _activations((t, n), gen, dev)).bfloat16() if case["residual"] else None
            state["dout"] = torch.randn((t, n), generator=gen, device=dev).bfloat16() if case["backward"] else None
    if "far" in state:  # the table that a program keeps: cos and sin of every position, [positions, rotary/2, 2]
        state["table"] = torch.stack(_cos_sin(torch.arange(state["far"], device=dev), case["rotary"], case["scaling"]), -1).float()
    return state


# -------------------------------------------------------------- plain forms


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    rstd = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + s["eps"])).float()
    y = h * rstd * s["weight"].float()
    out = {} if s["residual"] is None else {"sum": h.to(torch.bfloat16)}
    if c["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        out["y"] = _values(*_quantize(y, c["out"], s["gs"]), c["out"], s["gs"])
    return out


def _plain_rope(s):
    c = s["case"]
    cos, sin = s["table"][s["positions"]].unbind(-1)
    return _rotated(s["x"].float(), cos, -sin if c["backward"] else sin, c["rotary"], c["interleaved"]).to(torch.bfloat16)


def _plain_append(s):
    c, n = s["case"], s["real"]
    mode, page = c["mode"], c["page"]
    cos, sin = s["table"][s["positions"][:n]].unbind(-1)
    turn = lambda x: _rotated(x[:n].float(), cos, sin, c["rotary"], c["interleaved"])  # noqa: E731
    out = {"q": torch.cat([turn(s["q"]).to(torch.bfloat16), s["q_out"][n:]])}
    p, o = s["slot_map"][:n] // page, s["slot_map"][:n] % page
    for which, x in (("k", turn(s["k"])), ("v", s["v"][:n].float())):
        codes, scales = _quantize(x, mode, s["gs_" + which])
        s[which + "_codes"][p, :, o] = codes
        s[which + "_scales"][p, :, o] = scales
        out[which] = _values(s[which + "_codes"], s[which + "_scales"], mode, s["gs_" + which])
    return out


def _plain_sort(s):
    c = s["case"]
    ids, experts = s["ids"].flatten().long(), c["experts"]
    valid = (ids >= 0) & (ids < experts)
    key, order = torch.sort(torch.where(valid, ids, experts), stable=True)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=ids.device)
    return {"lhs_idx": torch.where(key < experts, order // c["k"], 0).int(), "rhs_idx": key.clamp(max=experts - 1).int(),
            "slot": torch.where(valid, slot, -1).int().view(s["ids"].shape),
            "offsets": torch.searchsorted(key, torch.arange(experts + 1, device=ids.device)).int()}


def _plain_combine(s):
    slot, w = s["slot"], s["weights"]
    valid = slot >= 0
    at = slot.clamp(min=0).long()
    if s["dout"] is None:
        y = torch.where(valid[..., None], s["y"][at].float(), 0.0)
        out = (y if w is None else y * w[..., None]).sum(1)
        return (out if s["residual"] is None else out + s["residual"].float()).to(torch.bfloat16)
    g = s["dout"].float()[:, None]
    t, k = slot.shape
    rows = torch.zeros_like(s["y"])
    dy = (g.expand(t, k, -1) if w is None else g * w[..., None]).to(torch.bfloat16)
    # rows of no token go behind the others and are cut off
    rows = torch.cat([rows, rows[:1]])
    rows[torch.where(valid, at, t * k).flatten()] = dy.flatten(0, 1)
    out = {"dy": rows[:-1]}
    if w is not None:
        out["dweights"] = torch.where(valid, (s["y"][at].float() * g).sum(-1), 0.0)
    return out


# --------------------------------------------------------------------- run


def _own_rope(s):
    from block_scaled_fp4_fp_gb300 import binding as B
    if "rope" not in s:
        c = s["case"]
        factor, original, low, high = _SCALING[c["scaling"]]
        s["rope"] = B.rope_table(s["far"], c["rotary"], base=_BASE, interleaved=c["interleaved"], scaling=c["scaling"],
                                 factor=factor, original_positions=original, low=low, high=high)
    return s["rope"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"norm": _plain_norm, "rope": _plain_rope, "append": _plain_append, "sort": _plain_sort,
                "combine": _plain_combine}[op](s)
    from block_scaled_fp4_fp_gb300 import binding as B
    mode = {"nvfp4": B.MODE_NVFP4, "mxfp4": B.MODE_MXFP4}.get(c.get("mode") or c.get("out"))
    if op == "norm":
        layout = B.SCALES_TILED if c["tiled"] else B.SCALES_LINEAR
        r = B.rms_norm(s["x"], s["weight"], eps=s["eps"], residual=s["residual"], mode=mode, global_scale=s["gs"], layout=layout)
        y = r.out
        if mode is not None:
            y = B.fp4_dequantize(r.xq, r.scales, mode=mode, global_scale=s["gs"], layout=layout)
        return {"y": y} if s["residual"] is None else {"sum": r.sum, "y": y}
    if op == "rope":
        return B.rope(_own_rope(s), s["x"], s["positions"], backward=c["backward"])
    if op == "append":
        if "cache" not in s:
            s["cache"] = B.kv_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], mode, s["gs_k"], s["gs_v"])
        B.kv_append_rope(s["cache"], _own_rope(s), s["k"], s["v"], s["slot_map"], s["positions"], q=s["q"], q_out=s["q_out"])
        out = {"q": s["q_out"]}
        for which in ("k", "v"):  # the cache is four matrices of the framework's formats: its own call reads them
            codes, scales = s[which + "_codes"], s[which + "_scales"]
            out[which] = B.fp4_dequantize(codes.view(-1, codes.shape[-1]), scales.view(-1, scales.shape[-1]), mode=mode,
                                          global_scale=s["gs_" + which]).view(*codes.shape[:-1], -1)
        return out
    if op == "sort":
        r = B.moe_sort(s["ids"], c["experts"])
        return {"lhs_idx": r.lhs_idx, "rhs_idx": r.rhs_idx, "slot": r.slot, "offsets": r.offsets}
    if s["dout"] is None:
        return B.moe_combine(s["y"], s["slot"], s["weights"], residual=s["residual"])
    dy, dweights = B.moe_combine_backward(s["dout"], s["slot"], s["weights"], y=s["y"] if c["weights"] else None,
                                          offsets=s["offsets"])
    return {"dy": dy} if dweights is None else {"dy": dy, "dweights": dweights}


# ---------------------------------------------------------- work and exact


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        a = 2 * n * (3 if case["residual"] else 1) + 2 * case["cols"]  # x; the residual, and the sum out
        if case["out"] == "bf16":
            return {"bytes": a + 2 * n, "flops": 5 * n}
        return {"bytes": a + 2 * n * (0.5 + 1 / _GROUP[case["out"]]) + 2 * n, "flops": 5 * n}  # and read back as values
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] * (1 + case["rotary"]), "flops": 3 * n * case["rotary"]}
    if op == "append":
        t, kv, heads, dim = sum(_lengths(case)[1]), case["kv_heads"], case["q_heads"], case["dim"]
        row = dim / 2 + dim / _GROUP[case["mode"]]  # bytes of one cached row
        rows = _cache_pages(case) * case["page"]
        # q read and written, new rows read and written; the whole cache read once and its values written
        return {"bytes": t * (4 * heads * dim + 2 * kv * (2 * dim + row) + 4 * case["rotary"] + 12)
                + 2 * kv * rows * (row + 2 * dim), "flops": 3 * t * (heads + kv) * case["rotary"]}
    t, k, e = case["tokens"], case["k"], case["experts"]
    if op == "sort":
        return {"bytes": 16 * t * k + 4 * (e + 1), "flops": 0}
    n, live = case["cols"], (t - case["pad"]) * k
    if case["backward"]:
        w = case["weights"]
        return {"bytes": 2 * n * (t - case["pad"]) + 2 * n * t * k + (2 * n * live if w else 0) + 4 * t * k * (3 if w else 1),
                "flops": (3 if w else 0) * live * n}
    return {"bytes": 2 * n * (live + t * (2 if case["residual"] else 1)) + t * k * (8 if case["weights"] else 4),
            "flops": 2 * live * n}


def _exact_grid(x, grid):
    """Nearest of the sorted grid's values to each |x| (ties to the even place), with x's sign."""
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
    lo = hi - 1
    below, above = a - grid[lo], grid[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(torch.signbit(x), -1.0, 1.0) * grid[torch.where(up, hi, lo)]


def _exact_quantized(x, mode, gs):
    """The values that x [..., D] in 64 bits is held as."""
    dev, g = x.device, _GROUP[mode]
    e2m1 = torch.tensor(_E2M1[:8], dtype=torch.float64, device=dev)
    x = x.reshape(*x.shape[:-1], -1, g)
    top = x.abs().amax(-1, keepdim=True)
    if mode == "nvfp4":
        e4m3 = torch.tensor(sorted([m * 2.0 ** -9 for m in range(8)]
                                   + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])[:-1],
                            dtype=torch.float64, device=dev)
        one = 1.0 if gs is None else gs.double()
        step = _exact_grid(top / (6 * one), e4m3) * one
    else:
        step = torch.where(top > 0, torch.ldexp(torch.ones_like(top), torch.frexp(top).exponent - 3), 2.0 ** -127)
    return torch.where(step > 0, _exact_grid(x / step.clamp(min=1e-300), e2m1) * step, 0.0).flatten(-2)


def _exact_stored(codes, scales, mode, gs):
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


def _exact_turned(x, positions, case, sign):
    """Each pair as a complex number times e^(i angle)."""
    rotary = case["rotary"]
    f, scale = _frequencies(rotary, case["scaling"])
    angle = positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    w = torch.polar(torch.full_like(angle, scale), sign * angle)[:, None]
    out = x.double().clone()
    half = rotary // 2
    first, second = ((slice(0, rotary, 2), slice(1, rotary, 2)) if case["interleaved"]
                     else (slice(0, half), slice(half, rotary)))
    z = torch.complex(out[..., first], out[..., second]) * w
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    if case["op"] == "sort":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out["sum"] = h
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["cols"] + s["eps"]) * s["weight"].double()
        out["y"] = y if case["out"] == "bf16" else _exact_quantized(y, case["out"], s["gs"])
        return out
    if case["op"] == "rope":
        return _exact_turned(s["x"], s["positions"], case, -1.0 if case["backward"] else 1.0)
    if case["op"] == "append":
        n, page = s["real"], case["page"]
        turned = {w: _exact_turned(s[w][:n], s["positions"][:n], case, 1.0) for w in "qk"}
        out = {"q": s["q_out"].double()}
        out["q"][:n] = turned["q"]
        for which, x in (("k", turned["k"]), ("v", s["v"][:n].double())):
            whole = _exact_stored(s[which + "_codes"], s[which + "_scales"], case["mode"], s["gs_" + which])
            whole[s["slot_map"][:n] // page, :, s["slot_map"][:n] % page] = _exact_quantized(x, case["mode"], s["gs_" + which])
            out[which] = whole
        return out
    t, k = s["slot"].shape
    valid, at = s["slot"] >= 0, s["slot"].clamp(min=0).long()
    w = torch.where(valid, 1.0 if s["weights"] is None else s["weights"].double(), 0.0).double()
    if s["dout"] is None:
        out = torch.zeros((t, case["cols"]), dtype=torch.float64, device=w.device)
        if s["residual"] is not None:
            out += s["residual"].double()
        for i in range(k):
            out += w[:, i, None] * s["y"][at[:, i]].double()
        return out
    g = s["dout"].double()
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=w.device)
    dw = torch.zeros_like(w)
    for i in range(k):
        dy.index_add_(0, at[:, i], w[:, i, None] * g)
        dw[:, i] = torch.where(valid[:, i], (g * s["y"][at[:, i]].double()).sum(-1), 0.0)
    return {"dy": dy} if s["weights"] is None else {"dy": dy, "dweights": dw}
