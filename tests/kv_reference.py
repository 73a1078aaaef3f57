"""Plain 64-bit implementations of the paged-cache operators, and the inputs their tests share.

Nothing here uses the library: formats are decoded from their bit fields, the
quantizer is the oracle's."""
import math
import random

import numpy as np
import torch

import oracle
from block_scaled_fp4_fp_gb300 import synth

GROUP = {2: 16, 1: 32}  # mode -> elements per scale
_E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def values(codes: np.ndarray, scales: np.ndarray, mode: int, gs: float = 1.0) -> np.ndarray:
    """codes uint32 [..., D/8], scales uint8 [..., D/group] -> float64 [..., D]."""
    nib = np.stack([(codes >> np.uint32(4 * k)) & np.uint32(15) for k in range(8)], -1)
    v = _E2M1[nib.reshape(*codes.shape[:-1], -1)]
    b = scales.astype(np.int64)
    if mode == 2:
        e, m = (b >> 3) & 15, b & 7
        s = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    else:
        s = 2.0 ** (b - 127.0)
    return v * np.repeat(s, v.shape[-1] // s.shape[-1], axis=-1) * gs


def quantize(x: torch.Tensor, mode: int, gs: float = None):
    """bf16 x [rows, D] -> oracle codes uint32 [rows, D/8], scales uint8."""
    u = synth.to_u16(x)
    if mode == 2:
        return oracle.nvfp4_quantize(u, np.float32(1.0 if gs is None else gs))
    return oracle.mxfp4_quantize(u)


class Problem:
    """A paged cache of random rows and a step's queries, on the CPU.  Slots no
    request may see hold codes with NaN scales; table entries no query needs are -1."""

    def __init__(self, mode, dim, kv_heads, group, page, cached, new, window=0, gs=False, seed=0, q_std=1.5):
        rng = random.Random(seed)
        self.mode, self.dim, self.kv_heads, self.q_heads, self.page = mode, dim, kv_heads, kv_heads * group, page
        self.cached, self.new, self.window = list(cached), list(new), window
        self.total = [a + b for a, b in zip(cached, new)]
        pages_of = [-(-n // page) for n in self.total]
        self.num_pages = sum(pages_of) + 3
        order = list(range(self.num_pages))
        rng.shuffle(order)
        self.max_pages = max(1, max(pages_of)) + 1
        table = np.full((len(cached), self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(pages_of):
            table[b, :n] = order[at:at + n]
            at += n
            if window and self.new[b]:  # pages behind every query's window have been given away
                first = max(0, self.total[b] - self.new[b] + 1 - window)
                table[b, :first // page] = -1
        self.table = table
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        tokens = int(self.starts[-1])
        self.gs_k = self.gs_v = None
        pool = 512
        raw = {}
        self.codes, self.scales = {}, {}
        g = np.random.RandomState(seed + 1)
        for w, std in (("k", 1.0), ("v", 0.7)):
            x = synth.bf16_normal((pool, dim), std, seed=seed * 7 + ord(w))
            x[:, :2] *= 4
            raw[w] = x
            gsv = float(np.float32(x.abs().max().item()) / np.float32(2688)) if gs else None
            setattr(self, "gs_" + w, gsv)
            c, s = quantize(x, mode, gsv)
            pick = g.randint(0, pool, (self.num_pages, kv_heads, page))
            self.codes[w], self.scales[w] = c[pick], s[pick].copy()
            self.scales[w][self.unseen()] = 0x7F if mode == 2 else 0xFF
        self.q = synth.bf16_normal((max(tokens, 1), self.q_heads, dim), q_std, seed=seed + 3)[:tokens]

    def unseen(self):
        """Boolean [pages, heads, slots]: True where no query may look."""
        m = np.ones((self.num_pages, self.kv_heads, self.page), bool)
        for b, n in enumerate(self.total):
            if not self.new[b]:
                continue
            lo = max(0, n - self.new[b] + 1 - self.window) if self.window else 0
            j = np.arange(lo, n)
            m[self.table[b, j // self.page], :, j % self.page] = False
        return m

    def cuda(self, B):
        dev = "cuda"
        t = {}
        for w in "kv":
            t[w + "c"] = torch.from_numpy(self.codes[w].view(np.int32).copy()).to(dev)
            t[w + "s"] = torch.from_numpy(self.scales[w].copy()).to(dev)
            gs = getattr(self, "gs_" + w)
            t["g" + w] = None if gs is None else torch.tensor(gs, dtype=torch.float32, device=dev)
        cache = B.kv_cache(t["kc"], t["ks"], t["vc"], t["vs"], self.mode, t["gk"], t["gv"])
        return cache, dict(q=self.q.to(dev), query_start=torch.from_numpy(self.starts).to(dev),
                           total_lens=torch.tensor(self.total, dtype=torch.int32, device=dev),
                           block_table=torch.from_numpy(self.table).to(dev))

    def attention(self, scale=None):
        """(out, lse, bound) in 64 bits: bound is how far a kernel may be from out at each element (see the
        attention tests for its derivation)."""
        scale = self.dim ** -0.5 if scale is None else scale
        out = np.zeros((self.q.shape[0], self.q_heads, self.dim))
        bound = np.zeros_like(out)
        lse = np.full(out.shape[:2], -np.inf)
        group = self.q_heads // self.kv_heads
        q = self.q.double().numpy()
        for b, n in enumerate(self.total):
            if not self.new[b]:
                continue
            lo = max(0, n - self.new[b] + 1 - self.window) if self.window else 0
            j = np.arange(lo, n)
            pg, sl = self.table[b, j // self.page], j % self.page
            for h in range(self.kv_heads):
                k = values(self.codes["k"][pg, h, sl], self.scales["k"][pg, h, sl], self.mode, np.float64(np.float32(self.gs_k or 1)))
                v = values(self.codes["v"][pg, h, sl], self.scales["v"][pg, h, sl], self.mode, np.float64(np.float32(self.gs_v or 1)))
                k1 = np.abs(k).sum(-1).max(initial=0.0)
                for i in range(self.new[b]):
                    t = self.starts[b] + i
                    pos = n - self.new[b] + i
                    see = j <= pos
                    if self.window:
                        see &= j > pos - self.window
                    if not see.any():
                        continue
                    qq = q[t, h * group:(h + 1) * group]
                    s = qq @ k[see].T * scale
                    m = s.max(-1, keepdims=True)
                    p = np.exp(s - m)
                    l = p.sum(-1, keepdims=True)
                    hs = slice(h * group, (h + 1) * group)
                    out[t, hs] = p @ v[see] / l
                    lse[t, hs] = (m + np.log(l))[:, 0]
                    ds = 2.0 ** -16 * np.abs(qq).max(-1, keepdims=True) * k1 * scale
                    bound[t, hs] = 2.0 ** -8 * np.abs(out[t, hs]) + ((1 + 2.0 ** -8) * np.exp(np.minimum(2 * ds, 700)) - 1) * (p @ np.abs(v[see]) / l) + 2.0 ** -126
        return out, lse, bound

    def lse_bound(self, scale=None):
        scale = self.dim ** -0.5 if scale is None else scale
        k = np.nan_to_num(values(self.codes["k"], self.scales["k"], self.mode, self.gs_k or 1))
        k[self.unseen()] = 0
        k1 = np.abs(k).sum(-1).max()
        return 2.0 ** -16 * np.abs(self.q.double().numpy()).max(-1) * k1 * scale + 2.0 ** -14


def plan(cached, new, free, table, page, tokens):
    """kv_plan on the host, token by token."""
    table = table.copy()
    slots, pos = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int32)
    start, taken, t = [0], 0, 0
    for b, (c, n) in enumerate(zip(cached, new)):
        for j in range(-(-c // page), -(-(c + n) // page)):
            table[b, j] = free[taken]
            taken += 1
        for i in range(n):
            p = c + i
            slots[t], pos[t] = int(table[b, p // page]) * page + p % page, p
            t += 1
        start.append(t)
    return table, np.array([a + b for a, b in zip(cached, new)], np.int32), np.array(start, np.int32), slots, pos, taken
