"""A decoder layer with experts, in 4 bits, as a server runs it: prompts of several lengths go in together, then every
request gets one token a step, from a captured graph that is padded to a fixed number of tokens.

    python examples/decoder_layer.py [--mode nvfp4|mxfp4] [--prompts 700 64 1] [--steps 32] [--check]

A step is: rms_norm, quantized on the way out -> qqmm (q, k, v) -> kv_plan -> kv_append_rope (K rotated and quantized
into the cache, q rotated in place) -> kv_attention -> qmm -> rms_norm with the residual -> router -> moe_sort ->
gather_qmm (gate and up) -> silu(gate) up -> gather_qmm (down) -> moe_combine with the residual.  Weights and inputs are
random; the router's softmax and the activation are torch's.  --check compares every step's stages with 64 bits, and the
gradients of moe_combine after the prompts."""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_fp4_fp_gb300 import binding as B, build

MODES = {"nvfp4": B.MODE_NVFP4, "mxfp4": B.MODE_MXFP4}


def rel(got, want):
    """Relative error; a NaN among them is infinitely far off (max and comparisons would drop it)."""
    e = float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
    return e if math.isfinite(e) else math.inf


def further(got, base, want):
    """How much further from `want` got is than base."""
    e = rel(got, want)
    return e if e == math.inf else max(0.0, e - rel(base, want))


def gather(worst, found):
    for name, v in found.items():
        worst[name] = max(worst.get(name, 0.0), v)


def off_limits(worst):
    """Stages further off than bf16 results are (2^-8 at most), attention's 8-bit probabilities twice that; the 4-bit norm is
    no further from the exact rows than the quantizer's own codes of them are, but for a few blocks."""
    return [name for name, v in worst.items() if not v <= (2.0 ** -7 if name == "attention" else 2.0 ** -8)]


class Layer:
    """Weights, cache and page bookkeeping of one layer, for a fixed set of requests."""

    def __init__(self, a):
        self.mode, self.a = MODES[a.mode], a
        g = torch.Generator(device="cuda").manual_seed(a.seed)
        randn = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        two_level = self.mode == B.MODE_NVFP4

        def weight(n, k, layout=B.SCALES_LINEAR, experts=None):
            w = (randn((experts or 1) * n, k) * k ** -0.5).bfloat16()
            gs = B.fp4_amax_global_scale(w) if two_level and experts is None else None
            codes, scales = B.fp4_quantize(w, self.mode, global_scale=gs, layout=layout)
            if experts:
                codes, scales = codes.view(experts, n, -1), scales.view(experts, n, -1)
            return codes, scales, gs

        self.w_qkv = weight((a.heads + 2 * a.kv_heads) * a.head_dim, a.hidden, B.SCALES_TILED)
        self.w_o = weight(a.hidden, a.heads * a.head_dim)
        self.w_gate_up, self.w_down = weight(2 * a.expert_dim, a.hidden, experts=a.experts), weight(a.hidden, a.expert_dim, experts=a.experts)
        self.w_router = (randn(a.experts, a.hidden) * a.hidden ** -0.5).bfloat16()
        self.norms = [(1 + 0.1 * randn(a.hidden)).bfloat16() for _ in range(2)]
        # scales of the normed rows and of K and V: here from the range of random projections, in a model from calibration
        self.gs = torch.tensor(8.0 / 2688, device="cuda") if two_level else None
        pages = [-(-(p + a.steps) // a.page) for p in a.prompts]
        self.cache = B.kv_cache_empty(sum(pages) + 4, a.kv_heads, a.page, a.head_dim, self.mode, self.gs, self.gs)
        self.lens = torch.zeros(len(a.prompts), dtype=torch.int32, device="cuda")
        self.table = torch.zeros((len(a.prompts), max(pages)), dtype=torch.int32, device="cuda")
        self.order = torch.randperm(sum(pages) + 4, generator=g, device="cuda").int()
        self.taken = torch.zeros((), dtype=torch.int64, device="cuda")
        self.spread = torch.arange(self.order.numel(), device="cuda")
        # positions up to four times the trained context
        self.scaling = dict(base=10000.0, scaling="ramp", factor=4.0, original_positions=1024, low=1.0, high=32.0)
        self.rope = B.rope_table(max(a.prompts) + a.steps, a.rotary, **self.scaling)
        # one workspace for prompts and tokens
        self.ws = B.kv_attention_workspace(self.cache, len(a.prompts), a.heads, max(a.prompts))

    def step(self, x, new, longest, keep=None):
        """x [tokens, hidden], the residual stream: the requests' new rows one after the other, then padding."""
        a, mode, T = self.a, self.mode, x.shape[0]
        n1 = B.rms_norm(x, self.norms[0], mode=mode, global_scale=self.gs, layout=B.SCALES_TILED)
        w, s, gs = self.w_qkv
        qkv = B.qqmm(n1.xq, n1.scales, w, s, self.gs, gs, mode=mode).view(T, -1, a.head_dim)
        q, k, v = qkv.split([a.heads, a.kv_heads, a.kv_heads], 1)
        if keep is not None:
            keep["unturned"] = q.clone()
        free = self.order[(self.spread + self.taken) % self.order.numel()]
        plan = B.kv_plan(self.lens, new, free, self.table, a.page, T)
        B.kv_append_rope(self.cache, self.rope, k, v, plan.slot_map, plan.positions, q=q, q_out=q)
        att = B.kv_attention(self.cache, q, plan.query_start, plan.total_lens, self.table, self.ws, max_query_len=longest,
                             out=torch.zeros((T, a.heads, a.head_dim), dtype=torch.bfloat16, device="cuda"))  # (rows of padding are not written)
        self.lens.copy_(plan.total_lens)
        self.taken.add_(plan.pages_taken)
        w, s, gs = self.w_o
        o = B.qmm(att.view(T, -1), w, s, global_scale_w=gs, mode=mode)
        n2 = B.rms_norm(o, self.norms[1], residual=x)
        top = (n2.out @ self.w_router.T).float().topk(a.top_k)
        weights = torch.softmax(top.values, -1)
        ids = torch.where(plan.positions[:, None] < 0, -1, top.indices).int()  # padding goes to no expert
        route = B.moe_sort(ids, a.experts)
        w, s, _ = self.w_gate_up
        gate, up = B.gather_qmm(n2.out, route.lhs_idx, route.rhs_idx, w, s, mode=mode).float().chunk(2, -1)
        act = (torch.nn.functional.silu(gate) * up).bfloat16()
        w, s, _ = self.w_down
        rows = torch.arange(act.shape[0], dtype=torch.int32, device="cuda")
        y = B.gather_qmm(act, rows, route.rhs_idx, w, s, mode=mode)
        out = B.moe_combine(y, route.slot, weights, residual=n2.sum)
        if keep is not None:
            keep.update(x=x.clone(), n1=n1, q=q, att=att, o=o, n2=n2, plan=plan, ids=ids, route=route, weights=weights, y=y, out=out)
        return out

    def check(self, k):
        """How far a step's stages are from 64 bits: the largest relative errors by name."""
        a, T, off = self.a, k["x"].shape[0], {}
        norm = lambda h, w: h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.double()  # noqa: E731
        # the first norm's codes are the quantizer's of the exact rows, but for blocks next to a border
        y = norm(k["x"].double(), self.norms[0])
        codes, scales = B.fp4_quantize(y.bfloat16(), self.mode, global_scale=self.gs, layout=B.SCALES_TILED)
        read = lambda c, s: B.fp4_dequantize(c, s, mode=self.mode, global_scale=self.gs, layout=B.SCALES_TILED).double()  # noqa: E731
        off["norm to 4 bits"] = further(read(k["n1"].xq, k["n1"].scales), read(codes, scales), y)
        h = k["o"].double() + k["x"].double()
        off["residual"], off["norm"] = rel(k["n2"].sum, h), rel(k["n2"].out, norm(h, self.norms[1]))
        # rotary positions of q
        pos = k["plan"].positions
        real = pos >= 0
        f, scale = B.rope_frequencies(a.rotary, **self.scaling)
        angle = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full_like(angle, scale), angle)[:, None]
        q, half = k["unturned"].double(), a.rotary // 2
        z = torch.complex(q[..., :half], q[..., half:a.rotary]) * turn
        want = torch.cat([z.real, z.imag, q[..., a.rotary:]], -1)
        off["rope"] = rel(k["q"][real], want[real])
        # attention over what the cache holds
        kc, ks, vc, vs, gk, gv = self.cache.tensors
        rows = lambda c, s, g: B.fp4_dequantize(c.view(-1, c.shape[-1]), s.view(-1, s.shape[-1]), mode=self.mode,  # noqa: E731
                                                global_scale=g).double().view(-1, a.kv_heads, a.page, a.head_dim)
        keys, vals, group = rows(kc, ks, gk), rows(vc, vs, gv), a.heads // a.kv_heads
        start, total, worst = k["plan"].query_start.tolist(), k["plan"].total_lens.tolist(), 0.0
        for b, n in enumerate(total):
            t = torch.arange(n, device="cuda")
            page, slot = self.table[b, t // a.page].long(), t % a.page
            kk, vv = (m[page, :, slot].repeat_interleave(group, 1) for m in (keys, vals))
            mine = slice(start[b], start[b + 1])
            score = torch.einsum("thd,nhd->htn", k["q"][mine].double(), kk) * a.head_dim ** -0.5
            last = n - (start[b + 1] - start[b]) + torch.arange(start[b + 1] - start[b], device="cuda")
            score.masked_fill_(t[None, None] > last[None, :, None], float("-inf"))
            worst = max(worst, rel(k["att"][mine], torch.einsum("htn,nhd->thd", score.softmax(-1), vv)))
        off["attention"] = worst
        # routing and the way back
        route, key = k["route"], torch.where(k["ids"] < 0, a.experts, k["ids"]).flatten()
        key, order = torch.sort(key, stable=True)
        kept = int((key < a.experts).sum())
        right = torch.equal(route.lhs_idx[:kept].long(), order[:kept] // a.top_k) and torch.equal(route.rhs_idx[:kept], key[:kept].int())
        right &= int(route.offsets[-1]) == kept and bool((route.slot.flatten()[order[:kept]] == torch.arange(kept, device="cuda")).all())
        off["sort"] = 0.0 if right else float("inf")
        w = torch.where(route.slot < 0, 0.0, k["weights"]).double()
        y = k["y"].double()[route.slot.clamp(min=0).long()]
        off["combine"] = rel(k["out"], k["n2"].sum.double() + (w[..., None] * y).sum(1))
        return off

    def gradients(self, k):
        """The same for the gradients of moe_combine, by the experts' rows and by the router's weights."""
        route, dout = k["route"], torch.randn(k["out"].shape, device="cuda").bfloat16()
        dy, dw = B.moe_combine_backward(dout, route.slot, k["weights"], y=k["y"], offsets=route.offsets)
        y, w = k["y"].double().requires_grad_(), k["weights"].double().requires_grad_()
        live = route.slot >= 0
        picked = torch.where(live[..., None], y[route.slot.clamp(min=0).long()], 0.0)
        ((w[..., None] * picked).sum(1) * dout.double()).sum().backward()
        return {"rows' gradient": rel(dy, y.grad), "weights' gradient": rel(dw, w.grad)}


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--mode", choices=MODES, default="nvfp4")
    p.add_argument("--prompts", type=int, nargs="+", default=[700, 64, 1, 1500])
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--hidden", type=int, default=5120)
    p.add_argument("--heads", type=int, default=40)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--rotary", type=int, default=128)
    p.add_argument("--page", type=int, default=64)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--top-k", type=int, default=4)
    p.add_argument("--expert-dim", type=int, default=2880)
    p.add_argument("--pad", type=int, default=3, help="tokens of padding in the captured step")
    p.add_argument("--seed", type=int, default=0)
    p.add_argument("--check", action="store_true")
    a = p.parse_args()
    build.build()
    B.fp4_init(0)
    layer, n, worst = Layer(a), len(a.prompts), {}

    # prompts
    x = torch.randn((sum(a.prompts), a.hidden), device="cuda").bfloat16()
    keep = {}
    layer.step(x, torch.tensor(a.prompts, dtype=torch.int32, device="cuda"), max(a.prompts), keep)
    if a.check:
        gather(worst, layer.check(keep))
        gather(worst, layer.gradients(keep))
    # tokens: one step runs eagerly, the others from a graph
    x = torch.randn((n + a.pad, a.hidden), device="cuda").bfloat16()
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, one, 1, keep)
    torch.cuda.current_stream().wait_stream(side)
    if a.check:
        gather(worst, layer.check(keep))
    keep, graph = {} if a.check else None, torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(x, one, 1, keep)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    for i in range(a.steps - 1):
        if a.check and i:
            x.copy_(y)
        graph.replay()
        if a.check:
            gather(worst, layer.check(keep))
    ev[1].record()
    torch.cuda.synchronize()
    status = B.fp4_check_device_error()
    if status != B.FP4_OK:
        raise SystemExit(f"device error: {B.status_string(status)}")
    want = [p + a.steps for p in a.prompts]
    if layer.lens.tolist() != want:
        raise SystemExit(f"lengths {layer.lens.tolist()}, expected {want}")
    if a.check:
        for name, v in worst.items():
            print(f"largest relative error, {name}: {v:.2e}")
        if off_limits(worst):
            raise SystemExit("off: " + ", ".join(off_limits(worst)))
    else:
        print(f"{n} requests, {sum(want)} tokens cached: {ev[0].elapsed_time(ev[1]) / max(a.steps - 1, 1) * 1e3:.1f} us a step")
    print("ok")


if __name__ == "__main__":
    main()
