"""A decoder's attention block over a paged 4-bit cache, as a server runs it: prompts of several lengths go in together,
then every request gets one token a step, from a captured graph.

    python examples/kv_decode.py [--mode nvfp4|mxfp4] [--prompts 700 64 1] [--steps 64] [--check]

A step is: projections (qmm over 4-bit weights) -> kv_plan (pages and slots for the new tokens) -> kv_append
(K and V quantized into them) -> kv_attention -> output projection.  Weights and inputs are random.  --check
compares every step with attention in 64 bits over the dequantized cache.  (Rotary positions: kv_append_rope in place of
kv_append, with kv_plan's positions; decoder_layer.py beside this file does so.)"""
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


class Block:
    """Weights, cache and page bookkeeping of one layer's attention, for a fixed set of requests."""

    def __init__(self, a):
        self.mode, self.heads, self.kv_heads, self.dim, self.page = MODES[a.mode], a.heads, a.kv_heads, a.head_dim, a.page
        g = torch.Generator(device="cuda").manual_seed(a.seed)
        rows = (a.heads + 2 * a.kv_heads) * a.head_dim

        def weight(n, k):
            w = (torch.randn((n, k), generator=g, device="cuda") * k ** -0.5).bfloat16()
            gs = None
            if self.mode == B.MODE_NVFP4:
                gs = B.fp4_amax_global_scale(w)
            codes, scales = B.fp4_quantize(w, self.mode, global_scale=gs)
            return codes, scales, gs

        self.w_qkv, self.w_o = weight(rows, a.hidden), weight(a.hidden, a.heads * a.head_dim)
        n = len(a.prompts)
        pages = [-(-(p + a.steps) // a.page) for p in a.prompts]
        # a global scale for K and V: here from the range of random projections, in a model from calibration
        gs = torch.tensor(8.0 / 2688, device="cuda") if self.mode == B.MODE_NVFP4 else None
        self.cache = B.kv_cache_empty(sum(pages) + 4, a.kv_heads, a.page, a.head_dim, self.mode, gs, gs)
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.table = torch.zeros((n, max(pages)), dtype=torch.int32, device="cuda")
        self.order = torch.randperm(sum(pages) + 4, generator=g, device="cuda").int()  # the pool's free pages
        self.taken = torch.zeros((), dtype=torch.int64, device="cuda")
        self.spread = torch.arange(self.order.numel(), device="cuda")

    def workspace(self, tokens):
        return B.kv_attention_workspace(self.cache, self.lens.numel(), self.heads, tokens)

    def step(self, x, new, ws, longest, keep=None):
        """x [tokens, hidden]: the requests' new rows one after the other, new[b] of them each."""
        w, s, gs = self.w_qkv
        qkv = B.qmm(x, w, s, global_scale_w=gs, mode=self.mode).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        free = self.order[(self.spread + self.taken) % self.order.numel()]
        plan = B.kv_plan(self.lens, new, free, self.table, self.page, x.shape[0])
        B.kv_append(self.cache, k, v, plan.slot_map)
        out = B.kv_attention(self.cache, q, plan.query_start, plan.total_lens, self.table, ws, max_query_len=longest)
        self.lens.copy_(plan.total_lens)
        self.taken.add_(plan.pages_taken)
        w, s, gs = self.w_o
        y = B.qmm(out.view(x.shape[0], -1), w, s, global_scale_w=gs, mode=self.mode)
        if keep is not None:
            keep.update(q=q, out=out, plan=plan)
        return y

    def exact(self, q, plan):
        """The attention of the last step in 64 bits over what the cache holds."""
        kc, ks, vc, vs, gs_k, gs_v = self.cache.tensors
        rows = lambda c, s, gs: B.fp4_dequantize(c.view(-1, c.shape[-1]), s.view(-1, s.shape[-1]), mode=self.mode,
                                                 global_scale=gs).double().view(-1, self.kv_heads, self.page, self.dim)
        keys, vals = rows(kc, ks, gs_k), rows(vc, vs, gs_v)
        out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        start, total = plan.query_start.tolist(), plan.total_lens.tolist()
        group = self.heads // self.kv_heads
        for b, n in enumerate(total):
            t = torch.arange(n, device="cuda")
            page, slot = self.table[b, t // self.page].long(), t % self.page
            k = keys[page, :, slot].repeat_interleave(group, 1)  # [n, heads, dim]
            v = vals[page, :, slot].repeat_interleave(group, 1)
            mine = slice(start[b], start[b + 1])
            score = torch.einsum("thd,nhd->htn", q[mine].double(), k) * self.dim ** -0.5
            last = n - (start[b + 1] - start[b]) + torch.arange(start[b + 1] - start[b], device="cuda")
            score.masked_fill_(t[None, None] > last[None, :, None], float("-inf"))
            out[mine] = torch.einsum("htn,nhd->thd", score.softmax(-1), v)
        return out


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--mode", choices=MODES, default="nvfp4")
    p.add_argument("--prompts", type=int, nargs="+", default=[700, 64, 1, 1500])
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--hidden", type=int, default=5120)
    p.add_argument("--heads", type=int, default=40)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--page", type=int, default=64)
    p.add_argument("--seed", type=int, default=0)
    p.add_argument("--check", action="store_true")
    a = p.parse_args()
    build.build()
    B.fp4_init(0)
    block = Block(a)
    n = len(a.prompts)
    worst = 0.0

    def check(keep):
        nonlocal worst
        want = block.exact(keep["q"], keep["plan"])
        worst = max(worst, rel(keep["out"], want))

    # one workspace for prompts and tokens
    ws = block.workspace(max(a.prompts))
    # prompts
    x = torch.randn((sum(a.prompts), a.hidden), device="cuda").bfloat16()
    keep = {}
    block.step(x, torch.tensor(a.prompts, dtype=torch.int32, device="cuda"), ws, max(a.prompts), keep)
    if a.check:
        check(keep)
    # tokens: one step runs eagerly, the others from a graph
    x = torch.randn((n, a.hidden), device="cuda").bfloat16()
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, one, ws, 1, keep)
    torch.cuda.current_stream().wait_stream(side)
    if a.check:
        check(keep)
    keep, graph = {}, torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, one, ws, 1, keep)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    for i in range(a.steps - 1):
        if a.check and i:
            x.copy_(y)
        graph.replay()
        if a.check:
            check(keep)
    ev[1].record()
    torch.cuda.synchronize()
    status = B.fp4_check_device_error()
    if status != B.FP4_OK:
        raise SystemExit(f"device error: {B.status_string(status)}")
    want = [p + a.steps for p in a.prompts]
    if block.lens.tolist() != want:
        raise SystemExit(f"lengths {block.lens.tolist()}, expected {want}")
    if a.check:
        # bf16 results of 8-bit probabilities
        print(f"largest relative error of a step's attention: {worst:.2e}")
        if worst > 2.0 ** -7:
            raise SystemExit("attention is off")
    else:
        print(f"{n} requests, {sum(want)} tokens cached: {ev[0].elapsed_time(ev[1]) / max(a.steps - 1, 1) * 1e3:.1f} us a step")
    print("ok")


if __name__ == "__main__":
    main()
