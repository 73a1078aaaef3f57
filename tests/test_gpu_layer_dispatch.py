"""The kernels that rules on sizes choose where tokens are many: each against 64 bits, at sizes taken from the GPU's number of
SMs so that the rule falls the way it is meant to on any of them."""
import numpy as np
import pytest
import torch

import kv_reference as K
import layer_reference as R
from block_scaled_fp4_fp_gb300 import synth
from helpers import u8, u32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.fp4_init(0)
    return binding


@pytest.fixture(scope="module")
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def sample(rows, n=60):
    """Rows at both ends, around multiples of 128 and here and there."""
    g = np.random.RandomState(rows)
    return np.unique(np.clip(np.r_[0:n, rows - n:rows, 126:131, g.randint(0, rows, n)], 0, rows - 1))


# ---------------------------------------------------------------- rms_norm
Y = 5 * 2.0 ** -24  # y before its rounding: h, 1/rms (its rounding, and half of a sum of squares that is off by less than 2^-23), two products


def many_rows(sms, cols):
    """More than 1024 chunks of 16 elements an SM: two chunks a thread."""
    return sms * 1024 // ((cols + 15) // 16) + 37


@pytest.mark.parametrize("cols", [24, 128, 264, 512, 1024, 2880, 5120])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_many_rows(B, sms, cols, residual):
    rows = many_rows(sms, cols)
    x, w = synth.bf16_normal((rows, cols), 1.0, seed=cols), (1 + 0.3 * synth.bf16_normal((1, cols), 1.0, seed=1).float()).bfloat16().view(-1)
    r = synth.bf16_normal((rows, cols), 3.0, seed=2) if residual else None
    got = B.rms_norm(x.cuda(), w.cuda(), residual=None if r is None else r.cuda())
    pick = sample(rows)
    h, y = R.rms_norm(x[pick], w, 1e-6, None if r is None else r[pick])
    R.assert_within(got.out[pick], y, Y * np.abs(y), "out")
    if residual:
        R.assert_within(got.sum[pick], h, 2.0 ** -24 * np.abs(h), "sum")


@pytest.mark.parametrize("cols", [32, 96, 128, 512, 1024, 2880, 5120])
@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("layout", [0, 1])
def test_norm_of_many_rows_in_four_bits(B, sms, cols, mode, layout):
    rows = many_rows(sms, cols)
    x, w = synth.bf16_normal((rows, cols), 1.0, seed=cols), (1 + 0.3 * synth.bf16_normal((1, cols), 1.0, seed=1).float()).bfloat16().view(-1)
    r = synth.bf16_normal((rows, cols), 3.0, seed=2) if cols != 512 else None
    gs = float(np.float32(0.0071)) if mode == 2 else None
    got = B.rms_norm(x.cuda(), w.cuda(), residual=None if r is None else r.cuda(), mode=mode, layout=layout,
                     global_scale=None if gs is None else torch.tensor(gs, device="cuda"))
    pick, groups = sample(rows), cols // R.GROUP[mode]
    scales = u8(got.scales)
    if layout == 1:
        rr, cc = np.broadcast_arrays(pick[:, None], np.arange(groups)[None])
        scales = scales.reshape(-1)[((rr // 128) * ((groups + 3) // 4) + cc // 4) * 512 + (rr % 32) * 16 + ((rr % 128) // 32) * 4 + cc % 4]
    else:
        scales = scales[pick]
    y = R.rms_norm(x[pick], w, 1e-6, None if r is None else r[pick])[1]
    R.check_codes(u32(got.xq)[pick], scales, y, Y * np.abs(y), mode, 1.0 if gs is None else gs)


# -------------------------------------------------------------------- rope


def many_tokens(sms, units):
    """So many that a thread takes as many heads as it can."""
    return sms * 512 // units + 61


@pytest.mark.parametrize("dim,rotary", [(128, 128), (128, 64), (96, 24), (64, 20)])
@pytest.mark.parametrize("heads", [3, 13, 18])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_many_tokens(B, sms, dim, rotary, heads, interleaved):
    tokens = many_tokens(sms, 4)
    table, (freqs, scale) = B.rope_table(tokens + 9, rotary, interleaved=interleaved), B.rope_frequencies(rotary)
    qkv = synth.bf16_normal((tokens, heads + 2, dim), 1.0, seed=heads + dim).cuda()
    x, pos = qkv[:, 1:1 + heads], torch.arange(9, 9 + tokens, dtype=torch.int32, device="cuda")
    for backward in (False, True):
        got, pick = B.rope(table, x, pos, backward=backward), sample(tokens)
        want, bound = R.rope(x[pick].cpu().double().numpy(), pick + 9, freqs, scale, interleaved, backward)
        R.assert_within(got[pick], want, bound, "rope")
        # whole rows the same as few tokens on their own, whose heads are shared out otherwise; and in place
        few = B.rope(table, x[5:40].contiguous(), pos[5:40], backward=backward)
        assert torch.equal(got[5:40], few)
    before = qkv.clone()
    B.rope(table, x, pos, backward=True, out=x)
    assert torch.equal(x, got) and torch.equal(qkv[:, 0], before[:, 0]) and torch.equal(qkv[:, -1], before[:, -1])


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary,kv,heads", [(128, 128, 5, 15), (128, 64, 3, 3), (64, 32, 8, 24), (96, 24, 3, 6), (32, 20, 2, 0), (256, 256, 1, 8)])
def test_append_of_many_tokens(B, sms, mode, interleaved, dim, rotary, kv, heads):
    page, tokens = 64, many_tokens(sms, dim // 16)
    pages = tokens // page + 2
    g = np.random.RandomState(dim + kv)
    slots, pos = g.permutation(pages * page)[:tokens].astype(np.int64), g.randint(0, 5000, tokens)
    slots[7], pos[7] = -1, -1
    slots[8] = -1
    table, (freqs, scale) = B.rope_table(5000, rotary, interleaved=interleaved), B.rope_frequencies(rotary)
    qkv = synth.bf16_normal((tokens, heads + 2 * kv, dim), 1.0, seed=dim).cuda()
    q, k, v = qkv.split([heads, kv, kv], 1)
    gs = [float(np.float32(0.0049)), float(np.float32(0.0031))] if mode == 2 else [None, None]
    cache = B.kv_cache_empty(pages, kv, page, dim, mode, *[None if s is None else torch.tensor(s, device="cuda") for s in gs])
    dpos = torch.from_numpy(pos).int().cuda()
    q_out = torch.full((tokens, heads, dim), 5.0, dtype=torch.bfloat16, device="cuda") if heads else None
    B.kv_append_rope(cache, table, k, v, torch.from_numpy(slots).cuda(), dpos, q=q if heads else None, q_out=q_out)
    assert B.fp4_check_device_error() == B.FP4_OK
    if heads:
        assert torch.equal(q_out, B.rope(table, q, dpos, out=torch.full_like(q_out, 5.0)))
    pick = sample(tokens)
    pick = pick[slots[pick] >= 0]
    words, groups = dim // 8, dim // B.GROUP[mode]
    at = tuple(torch.from_numpy(i).cuda() for i in (slots[pick] // page, slots[pick] % page))
    taken = [t[at[0], :, at[1]] for t in cache.tensors[:4]]
    y, dy = R.rope(k[pick].cpu().double().numpy(), pos[pick], freqs, scale, interleaved)
    R.check_codes(u32(taken[0]).reshape(-1, words), u8(taken[1]).reshape(-1, groups), y.reshape(-1, dim), dy.reshape(-1, dim), mode,
                  1.0 if gs[0] is None else gs[0])
    c, s = K.quantize(v[pick].reshape(-1, dim).contiguous().cpu(), mode, gs[1])
    assert np.array_equal(u32(taken[2]).reshape(-1, words), c.reshape(-1, words)) and np.array_equal(u8(taken[3]).reshape(-1, groups), s.reshape(-1, groups))
    # no slot beside the tokens'
    free = np.ones(pages * page, bool)
    free[slots[slots >= 0]] = False
    free = torch.from_numpy(free).cuda().view(pages, page)
    assert not any(t.transpose(1, 2)[free].any() for t in cache.tensors[:4])


# -------------------------------------------------------------------- moe
# (tokens a SM, k, cols): a warp a token, a small CTA a token, a large one; k of one batch of two, four or eight rows and of several
MANY = [(33, 2, 512), (33, 4, 1000), (33, 6, 512), (33, 11, 264), (5, 2, 2880), (5, 4, 2880), (5, 8, 1032), (5, 11, 264), (5, 1, 16), (4, 3, 4104), (9, 4, 1032),
        (1, 8, 2880), (1, 11, 4104)]


@pytest.mark.parametrize("per_sm,k,cols", MANY)
@pytest.mark.parametrize("weights", [False, True])
def test_combine_of_many_tokens(B, sms, per_sm, k, cols, weights):
    """Forward and gradients, from 64 bits on the GPU."""
    tokens = per_sm * sms + 3
    g = np.random.RandomState(cols + k)
    ids = np.minimum((32 * g.rand(tokens, k) ** 2).astype(np.int32), 31)
    ids[g.rand(tokens, k) < 0.1] = -1
    plan = B.moe_sort(torch.from_numpy(ids).cuda(), 32)
    kept, slot = int(plan.offsets[-1]), plan.slot
    y, dout, r = (synth.bf16_normal((n, cols), 1.0, seed=s).cuda() for n, s in ((tokens * k, 1), (tokens, 2), (tokens, 3)))
    w = torch.softmax(synth.bf16_normal((tokens, k), 1.0, seed=4).float(), -1).cuda() if weights else None
    live, at = slot >= 0, slot.clamp(min=0).long()
    wd = torch.ones((tokens, k), dtype=torch.float64, device="cuda") if w is None else w.double()
    want, size = r.double(), r.double().abs()
    dw, dsize = torch.zeros_like(wd), torch.zeros_like(wd)
    for j in range(k):
        row = torch.where(live[:, j, None], y[at[:, j]].double(), 0.0)
        want, size = want + wd[:, j, None] * row, size + (wd[:, j, None] * row).abs()
        dw[:, j], dsize[:, j] = (dout.double() * row).sum(1), (dout.double() * row).abs().sum(1)
    out = B.moe_combine(y, slot, w, residual=r)
    off = (out.double() - want).abs() - (2.0 ** -8 * (want.abs() + size * (k * 2.0 ** -24)) + size * (k * 2.0 ** -24))  # k + 1 terms in fp32, a rounding
    assert off.max() <= 0
    dy, dweights = B.moe_combine_backward(dout, slot, w, y=y, offsets=plan.offsets, dy=torch.full_like(y, 3.0))
    assert B.fp4_check_device_error() == B.FP4_OK
    # cols roundings of 2^-24 of the sum of absolute values at most
    assert ((dweights.double() - dw).abs() <= cols * 2.0 ** -24 * dsize).all() and (dweights[~live] == 0).all()
    for j in range(k):
        rows, mine = at[live[:, j], j], live[:, j]
        exact = wd[mine, j, None] * dout[mine].double()
        assert ((dy[rows].double() - exact).abs() <= (2.0 ** -8 + 2.0 ** -23) * exact.abs()).all()
    assert (dy[kept:] == 0).all()
    again = B.moe_combine_backward(dout, slot, w, y=y, offsets=plan.offsets)
    assert torch.equal(again[0], dy) and torch.equal(again[1], dweights)
    only, none = B.moe_combine_backward(dout, slot, w, offsets=plan.offsets)
    assert none is None and torch.equal(only, dy)
