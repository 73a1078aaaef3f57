"""kv_attention's scores, against 64 bits, where a channel of the queries is far above the others.

The scores are claimed to be fp32 sums of the exact products, but for what the few-row kernel leaves of a query,
2^-23 of the row's largest element.  A sum of at most 64 rounded partial sums (the tensor cores add 16 or 64 products at a
time, the other kernel one by one in groups of at most 32) is within 64 2^-24 of the sum of the magnitudes, so
    ds = scale (2^-18 max_j sum_d |q_d k_jd| + 2^-23 max|q| max_j |k_j|_1)
bounds a score's error, and, with A = sum_j p_j |v_j| / sum_j p_j and p in at least 8 significant bits,
    |out - exact| <= 2^-8 |exact| + ((1 + 2^-8) exp(2 ds) - 1) A + 2^-126 (1 + sum_j |v_j|)
    |lse - exact| <= ds + 2^-14
(what exp2, the sums of p and the last logarithm add is below 2^-14; 2^-126 is fp32's and bf16's smallest normal number,
below which outputs, and the p of the row's sum of at least 1, may be 0)."""
import numpy as np
import pytest
import torch

import kv_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.fp4_init(0)
    return binding


def check_tight(B, p, scale=None):
    cache, t = p.cuda(B)
    scale = p.dim ** -0.5 if scale is None else scale
    ws = B.kv_attention_workspace(cache, len(p.new), p.q_heads, max(p.new))
    sums = torch.empty((p.q.shape[0], p.q_heads), device="cuda")
    out = B.kv_attention(cache, t["q"], t["query_start"], t["total_lens"], t["block_table"], ws, max_query_len=max(p.new), scale=scale,
                         lse=sums)
    assert B.fp4_check_device_error() == B.FP4_OK
    got, lse = out.double().cpu().numpy(), sums.double().cpu().numpy()
    want, wlse, _ = p.attention(scale)
    group = p.q_heads // p.kv_heads
    bounds = np.zeros_like(want)
    q = p.q.double().numpy()
    for b, n in enumerate(p.total):
        j = np.arange(n)
        pg, sl = p.table[b, j // p.page], j % p.page
        for h in range(p.kv_heads):
            k, v = (np.abs(R.values(p.codes[w][pg, h, sl], p.scales[w][pg, h, sl], p.mode, np.float64(np.float32(gs or 1))))
                    for w, gs in (("k", p.gs_k), ("v", p.gs_v)))
            kv = R.values(p.codes["k"][pg, h, sl], p.scales["k"][pg, h, sl], p.mode, np.float64(np.float32(p.gs_k or 1)))
            for i in range(p.new[b]):
                t_, hs, see = p.starts[b] + i, slice(h * group, (h + 1) * group), n - p.new[b] + i + 1
                qq = q[t_, hs]
                ds = scale * (2.0 ** -18 * (np.abs(qq) @ k[:see].T).max(-1) + 2.0 ** -23 * np.abs(qq).max(-1) * k[:see].sum(-1).max())
                s = qq @ kv[:see].T * scale
                pr = np.exp(s - wlse[t_, hs][:, None])
                bound = (2.0 ** -8 * np.abs(want[t_, hs]) + ((1 + 2.0 ** -8) * np.exp(2 * ds)[:, None] - 1) * (pr @ v[:see])
                         + 2.0 ** -126 * (1 + v[:see].sum(0)))
                bounds[t_, hs] = bound
                assert (np.abs(got[t_, hs] - want[t_, hs]) <= bound).all(), \
                    f"token {t_}, kv head {h}: off by {np.abs(got[t_, hs] - want[t_, hs]).max():.3g} of {bound.max():.3g}"
                assert (np.abs(lse[t_, hs] - wlse[t_, hs]) <= ds + 2.0 ** -14).all()
    return np.median(bounds / np.abs(want).mean())


KERNELS = [  # dim, kv heads, group, queries: few rows (one block of eight, two), prompts, other head sizes
    (128, 2, 4, 1), (128, 1, 8, 2), (128, 1, 8, 9), (64, 2, 8, 1), (64, 1, 8, 3), (64, 1, 4, 20), (256, 1, 4, 1), (256, 1, 2, 9), (96, 1, 4, 2),
]


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,kv,group,new", KERNELS)
@pytest.mark.parametrize("large", [0.0, 2.0 ** 7, 2.0 ** 10, 2.0 ** 12, 2.0 ** 14])
def test_one_channel_of_the_queries_far_above_the_others(B, mode, dim, kv, group, new, large):
    """The keys are zero in that channel, so that the others decide."""
    p = R.Problem(mode, dim, kv, group, 64, [400, 33, 700], [new] * 3, gs=mode == 2, seed=dim + new)
    if large:
        p.q[..., 13] = torch.where(p.q[..., 13] < 0, -large, large).to(torch.bfloat16)
        p.codes["k"][..., 1] &= np.uint32(0xFF0FFFFF)
    check_tight(B, p)


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,new", [(128, 1), (64, 1), (256, 1), (128, 2), (128, 12), (64, 20), (96, 1)])
@pytest.mark.parametrize("below", [10.0, 20.0, 24.0, 28.5, 40.0, 100.0])
def test_small_probabilities_count_with_eight_bits(B, mode, dim, new, below):
    """One key `below` above the others in log2 has zeros for values in some channels: there the others decide, however small
    their probabilities are."""
    one_key_above(B, mode, dim, new, below)


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,new", [(128, 1), (64, 1), (256, 1), (128, 2)])
@pytest.mark.parametrize("below", [23.3, 23.6, 24.3, 24.6, 24.9, 25.1, 25.6])
def test_small_probabilities_at_the_end_of_f16(B, mode, dim, new, below):
    one_key_above(B, mode, dim, new, below)


def one_key_above(B, mode, dim, new, below):
    p = R.Problem(mode, dim, 1, 8, 64, [31 - new], [new], seed=dim + new)
    p.codes["k"][:] = 0
    p.scales["k"][..., 0] = 0x38 if mode == 2 else 127  # 1
    p.codes["k"][p.table[0, 0], 0, 0, 0] = 0x7  # 6 in channel 0 of key 0
    p.codes["v"][p.table[0, 0], 0, 0, 1:] = 0
    for w in "kv":
        p.scales[w][p.unseen()] = 0x7F if mode == 2 else 0xFF
    p.q[:] = 0
    p.q[..., 0] = below / 6 / 1.4426950408889634 * dim ** 0.5
    check_tight(B, p)


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,new", [(128, 1), (64, 1), (256, 1), (128, 2), (64, 9), (128, 30), (96, 2)])
@pytest.mark.parametrize("scale", [None, 3.0])
def test_sharp_and_rising_scores_closely(B, mode, dim, new, scale):
    """Scores that grow along the context, so that the references move, and that leave a few keys or one."""
    p = R.Problem(mode, dim, 1, 8, 64, [1500, 640], [new] * 2, seed=3, q_std=12.0)
    for b in range(2):
        j = np.arange(p.total[b])
        grow = 0x20 + 24 * j // p.total[b] if mode == 2 else 124 + 4 * j // p.total[b]
        p.scales["k"][p.table[b, j // 64], 0, j % 64] = grow[:, None].astype(np.uint8)
    assert check_tight(B, p, scale) < 0.5  # of the outputs' mean size: zeros would not pass
