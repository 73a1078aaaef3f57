"""Rotary tables, rope and kv_append_rope against 64 bits."""
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


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


SCALINGS = [dict(), dict(scaling="ramp", factor=16.0, original_positions=4096, low=1.0, high=32.0),
            dict(scaling="wavelength", factor=8.0, original_positions=8192, low=1.0, high=4.0)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("positions,rotary", [(1, 2), (131072, 64), (1 << 20, 8), (77, 256), (4097, 34)])
def test_table(B, positions, rotary, kw):
    """Each entry is the rounding of scale cos(angle): half a step, and the fp64 reference's own angle, off by 2^-53 of
    itself twice."""
    t = B.rope_table(positions, rotary, **kw).tensor
    freqs, scale = B.rope_frequencies(rotary, **kw)
    pick = np.unique(np.r_[0:min(positions, 300), np.random.RandomState(0).randint(0, positions, 2000), positions - 1])
    a = pick[:, None].astype(np.float64) * np.array(freqs)
    got = t.cpu().double().numpy()[pick]
    for i, want in ((0, np.cos(a) * scale), (1, np.sin(a) * scale)):
        assert np.all(np.abs(got[..., i] - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -52 * scale * (np.abs(a) + 1) + 2.0 ** -149)


def test_table_of_own_frequencies(B):
    """Frequencies above a turn a position, negative ones and zero; the scale counts."""
    f = [7.0, -0.3, 0.0, 1e-9]
    t = B.rope_table(1000, 8, frequencies=f, scale=0.75).tensor.cpu().double().numpy()
    a = np.arange(1000.0)[:, None] * np.array(f)
    for i, want in ((0, np.cos(a) * 0.75), (1, np.sin(a) * 0.75)):
        assert np.all(np.abs(t[..., i] - want) <= 2.0 ** -25 + 2.0 ** -52 * (np.abs(a) + 1))


# (dim, rotary): whole heads, halves and quarters in whole pieces; rotations that are no whole pieces
DIMS = [(64, 64), (128, 128), (128, 64), (256, 256), (256, 64), (96, 96), (8, 8), (16, 16), (80, 32), (96, 24), (64, 20), (8, 2), (40, 38),
        (128, 8)]


@pytest.mark.parametrize("dim,rotary", DIMS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_rope(B, dim, rotary, interleaved, backward):
    tokens, heads = 37, 5
    table = B.rope_table(9000, rotary, interleaved=interleaved, **SCALINGS[1])
    freqs, scale = B.rope_frequencies(rotary, **SCALINGS[1])
    g = np.random.RandomState(dim + rotary)
    pos = g.randint(0, 9000, tokens)
    pos[0], pos[1] = 0, 8999
    qkv = synth.bf16_normal((tokens, heads + 3, dim), 1.0, seed=dim + rotary).cuda()
    x = qkv[:, 2:2 + heads]
    want, bound = R.rope(x.cpu().double().numpy(), pos, freqs, scale, interleaved, backward)
    got = B.rope(table, x, ints(pos), backward=backward)
    assert got.is_contiguous()
    R.assert_within(got, want, bound, "rope")
    if rotary < dim:
        assert torch.equal(got[..., rotary:], x[..., rotary:])
    # into a view, and in place: the same bits, and nothing beside them
    wide = torch.full((tokens, heads + 2, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    B.rope(table, x, ints(pos), backward=backward, out=wide[:, 1:1 + heads])
    assert torch.equal(wide[:, 1:1 + heads], got) and (wide[:, 0] == 3).all() and (wide[:, -1] == 3).all()
    before = qkv.clone()
    assert B.rope(table, x, ints(pos), backward=backward, out=x) is x
    assert torch.equal(x, got) and torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 2 + heads:], before[:, 2 + heads:])
    assert B.fp4_check_device_error() == B.FP4_OK


@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 128), (1, 64, 128), (4000, 40, 128), (70000, 1, 16), (3, 300, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_sizes(B, tokens, heads, dim, interleaved):
    table = B.rope_table(tokens + 5, dim, interleaved=interleaved)
    freqs, scale = B.rope_frequencies(dim)
    x = synth.bf16_normal((tokens, heads, dim), 1.0, seed=tokens).cuda()
    pos = torch.arange(5, 5 + tokens, dtype=torch.int32, device="cuda")
    got = B.rope(table, x, pos)
    pick = np.unique(np.r_[0:min(tokens, 20), tokens // 2, max(0, tokens - 20):tokens])
    want, bound = R.rope(x[pick].cpu().double().numpy(), pick + 5, freqs, scale, interleaved)
    R.assert_within(got[pick], want, bound, "rope")


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_gradient_against_differences(B, interleaved):
    """The rotation is linear: <rope(x + d) - rope(x), g> = <d, backward(g)>.  Both sides' values are bf16 numbers, each
    off by 2^-8 of itself, which bounds the two sums' distance."""
    tokens, heads, dim = 9, 3, 64
    table = B.rope_table(500, 48, interleaved=interleaved, **SCALINGS[1])
    pos = ints(np.arange(7, 7 + tokens) * 31)
    x, d, g = (synth.bf16_normal((tokens, heads, dim), 1.0, seed=s).cuda() for s in (1, 2, 3))
    xd = (x.float() + d.float()).bfloat16()
    a, b, back = B.rope(table, xd, pos), B.rope(table, x, pos), B.rope(table, g, pos, backward=True)
    step = xd.double() - x.double()
    left, right = ((a.double() - b.double()) * g.double()).sum(), (step * back.double()).sum()
    bound = 2.0 ** -8 * (((a.double().abs() + b.double().abs()) * g.double().abs()).sum() + (step * back.double()).abs().sum()) * 1.01
    assert abs(left - right) <= bound


def test_padding_and_positions_past_the_table(B):
    table = B.rope_table(100, 64)
    x = synth.bf16_normal((6, 2, 64), 1.0, seed=1).cuda()
    for out in (None, x):
        y = torch.full_like(x, 9.0) if out is None else x.clone()
        src = x if out is None else y
        before = y.clone()
        B.rope(table, src, ints([3, -1, 99, 100, -2 ** 31, 2 ** 31 - 1]), out=y)
        assert B.fp4_check_device_error() == B.FP4_ERR_INVALID_ARG
        assert torch.equal(y[[1, 3, 4, 5]], before[[1, 3, 4, 5]]) and not torch.equal(y[[0, 2]], before[[0, 2]])
    B.rope(table, x, ints([-1] * 6), out=x)
    assert B.fp4_check_device_error() == B.FP4_OK


def test_a_callers_own_table(B):
    """A table the caller made, at an address of 8 bytes: the same bits as at one of 16."""
    for interleaved in (False, True):
        for rotary in (64, 20):
            made = B.rope_table(50, rotary, interleaved=interleaved)
            buf = torch.zeros(50 * rotary + 2, device="cuda")
            odd = buf[2:].view(50, rotary // 2, 2)
            odd.copy_(made.tensor)
            assert odd.data_ptr() % 16 == 8
            x, pos = synth.bf16_normal((50, 3, 64), 1.0, seed=5).cuda(), torch.arange(50, dtype=torch.int32, device="cuda")
            assert torch.equal(B.rope(made, x, pos), B.rope(B.rope_from_table(odd, interleaved), x, pos))


# ----------------------------------------------------------- kv_append_rope


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary,kv,heads,tokens,page", [(128, 128, 8, 64, 77, 64), (64, 32, 1, 8, 1, 16), (128, 64, 40, 40, 3, 128),
                                                             (32, 32, 3, 3, 65, 32), (256, 64, 2, 6, 130, 16), (96, 96, 5, 5, 33, 32),
                                                             (96, 24, 2, 4, 20, 16), (64, 38, 2, 2, 9, 64), (160, 16, 1, 1, 40, 32)])
def test_append_rope(B, mode, interleaved, dim, rotary, kv, heads, tokens, page):
    gs = mode == 2 and dim != 64
    pages = tokens // page + 3
    g = np.random.RandomState(tokens + dim)
    slots = g.permutation(pages * page)[:tokens].astype(np.int64)
    pos = g.randint(0, 5000, tokens)
    if tokens > 3:
        slots[2] = -1           # no room for this token: its q is rotated all the same
        slots[3], pos[3] = -1, -1  # padding
    table = B.rope_table(5000, rotary, interleaved=interleaved, **SCALINGS[2])
    freqs, scale = B.rope_frequencies(rotary, **SCALINGS[2])
    qkv = synth.bf16_normal((tokens, heads + 2 * kv, dim), 1.0, seed=dim + tokens)
    qkv[0, heads] = 0  # an all-zero K head
    q, k, v = qkv.split([heads, kv, kv], 1)
    gsv = [float(np.float32(0.0049)), float(np.float32(0.0031))] if gs else [None, None]
    words, groups = dim // 8, dim // B.GROUP[mode]
    old = [np.random.RandomState(5).randint(-2 ** 31, 2 ** 31, (pages, kv, page, words)).astype(np.int32),
           np.random.RandomState(6).randint(0, 256, (pages, kv, page, groups)).astype(np.uint8)]
    t = [torch.from_numpy(a.copy()).cuda() for a in (old[0], old[1], old[0], old[1])]
    cache = B.kv_cache(*t, mode, *[None if x is None else torch.tensor(x, device="cuda") for x in gsv])
    d = qkv.cuda()
    dq, dk, dv = d.split([heads, kv, kv], 1)
    q_out = torch.full((tokens, heads, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    assert B.kv_append_rope(cache, table, dk, dv, torch.from_numpy(slots).cuda(), ints(pos), q=dq, q_out=q_out) is q_out
    assert B.fp4_check_device_error() == B.FP4_OK
    # q: rope's bits; K and V: the rule's, and no slot beside them changed
    want_q = torch.full_like(q_out, 5.0)
    B.rope(table, dq, ints(pos), out=want_q)
    assert torch.equal(q_out, want_q)
    live = [i for i in range(tokens) if slots[i] >= 0]
    keep = np.ones((pages, kv, page), bool)
    keep[slots[live] // page, :, slots[live] % page] = False
    at = (slots[live] // page, slice(None), slots[live] % page)
    for x, gx, codes, scales, turned in ((k, gsv[0], t[0], t[1], True), (v, gsv[1], t[2], t[3], False)):
        codes, scales = u32(codes), u8(scales)
        assert np.array_equal(codes[keep], old[0].view(np.uint32)[keep]) and np.array_equal(scales[keep], old[1][keep])
        if turned:
            y, dy = R.rope(x.double().numpy()[live], pos[live], freqs, scale, interleaved)
            R.check_codes(codes[at].reshape(-1, words), scales[at].reshape(-1, groups), y.reshape(-1, dim), dy.reshape(-1, dim), mode,
                          1.0 if gx is None else gx)
        else:
            c, s = K.quantize(x.reshape(-1, dim).contiguous(), mode, gx)
            assert np.array_equal(codes[at], c.reshape(tokens, kv, words)[live]) and np.array_equal(scales[at], s.reshape(tokens, kv, groups)[live])
    # q in place, and no q at all: the same cache
    kept = [a.clone() for a in t]
    for a, b in zip(t, (old[0], old[1], old[0], old[1])):
        a.copy_(torch.from_numpy(b))
    B.kv_append_rope(cache, table, dk, dv, torch.from_numpy(slots).cuda(), ints(pos), q=dq, q_out=dq)
    rows = [i for i in range(tokens) if pos[i] >= 0]
    assert torch.equal(dq[rows], q_out[rows]) and all(torch.equal(a, b) for a, b in zip(t, kept))
    assert B.kv_append_rope(cache, table, dk, dv, torch.from_numpy(slots).cuda(), ints(pos)) is None
    assert all(torch.equal(a, b) for a, b in zip(t, kept))


@pytest.mark.parametrize("mode", [2, 1])
def test_without_a_turn_it_is_kv_append(B, mode):
    """cos 1 and sin 0: kv_append's bits, but for a zero's sign: (-0) 1 - b 0 is +0 where b is negative."""
    def unsigned_zeros(t):
        if t.dtype == torch.uint8:
            return t
        nib = torch.stack([(t >> (4 * i)) & 15 for i in range(8)])
        return torch.where(nib == 8, 0, nib)

    still = torch.zeros((50, 64, 2), device="cuda")
    still[..., 0] = 1
    k, v = (synth.bf16_normal((50, 4, 128), 1.0, seed=s).cuda() for s in (1, 2))
    k[3] *= 1e30
    k[4] *= 1e-38
    slots, pos = torch.arange(50, device="cuda"), torch.arange(50, dtype=torch.int32, device="cuda")
    a, b = (B.kv_cache_empty(2, 4, 32, 128, mode) for _ in range(2))
    B.kv_append(a, k, v, slots)
    for interleaved in (False, True):
        B.kv_append_rope(b, B.rope_from_table(still, interleaved), k, v, slots, pos)
        assert all(torch.equal(unsigned_zeros(x), unsigned_zeros(y)) for x, y in zip(a.tensors[:4], b.tensors[:4]))


def test_append_rope_skips_and_reports(B):
    table = B.rope_table(64, 64)
    k = synth.bf16_normal((4, 1, 64), 1.0, seed=1).cuda()
    for slots, pos in (([0, 32, 31, 2 ** 40], [5, 6, 7, 8]), ([0, 1, 31, 2], [5, 64, 7, 2 ** 31 - 1])):
        cache = B.kv_cache_empty(2, 1, 16, 64)
        q = torch.full((4, 1, 64), 4.0, dtype=torch.bfloat16, device="cuda")
        B.kv_append_rope(cache, table, k, k, torch.tensor(slots, device="cuda"), ints(pos), q=k, q_out=q)
        assert B.fp4_check_device_error() == B.FP4_ERR_INVALID_ARG
        codes = cache.tensors[0]
        assert codes[0, 0, 0].any() and codes[1, 0, 15].any() and int((codes != 0).any(-1).sum()) == 2
        assert (q[1] == 4).all().item() == (pos[1] == 64) and (q[3] == 4).all().item() == (pos[3] > 64)


def test_append_rope_from_a_graph_after_a_plan(B):
    """Positions and slots as kv_plan leaves them on the device, padding among them, in a captured step."""
    table = B.rope_table(400, 128)
    qkv = synth.bf16_normal((9, 6, 128), 1.0, seed=3).cuda()
    q, k, v = qkv.split([4, 1, 1], 1)
    caches, outs = [], []
    for captured in (False, True):
        cache = B.kv_cache_empty(12, 1, 16, 128)
        lens, new = ints([0, 15, 300]), ints([2, 3, 1])
        tbl = torch.zeros((3, 20), dtype=torch.int32, device="cuda")
        free = torch.arange(12, dtype=torch.int32, device="cuda").flip(0).contiguous()

        def step(out):
            plan = B.kv_plan(lens, new, free, tbl, 16, 9)
            B.kv_append_rope(cache, table, k, v, plan.slot_map, plan.positions, q=q, q_out=out)

        out = torch.zeros((9, 4, 128), dtype=torch.bfloat16, device="cuda")
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(out)
            graph.replay()
        else:
            step(out)
        assert B.fp4_check_device_error() == B.FP4_OK
        caches.append(cache)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and (outs[0][6:] == 0).all() and outs[0][:6].any()
    assert all(torch.equal(a, b) for a, b in zip(caches[0].tensors[:4], caches[1].tensors[:4]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_before_tokens(B, interleaved):
    """A [heads, tokens, head_dim] tensor seen as [tokens, heads, head_dim]."""
    table = B.rope_table(300, 64, interleaved=interleaved)
    x = synth.bf16_normal((6, 200, 96), 1.0, seed=4).cuda()
    pos = torch.arange(50, 250, dtype=torch.int32, device="cuda")
    want = B.rope(table, x.transpose(0, 1).contiguous(), pos)
    assert torch.equal(B.rope(table, x.transpose(0, 1), pos), want)
    B.rope(table, x.transpose(0, 1), pos, out=x.transpose(0, 1))
    assert torch.equal(x.transpose(0, 1), want)


def test_elements_past_32_bits(B):
    """A view of more than 2^31 elements, rotated in place."""
    tokens, heads, dim = 70000, 128, 256
    table = B.rope_table(tokens, 64)
    x = torch.zeros((tokens, heads, dim), dtype=torch.bfloat16, device="cuda")
    pick = torch.tensor([0, 65535, 65537, tokens - 1], device="cuda")
    part = synth.bf16_normal((4, heads, dim), 1.0, seed=5).cuda()
    x[pick] = part
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    B.rope(table, x, pos, out=x)
    assert torch.equal(x[pick], B.rope(table, part, pick.int()))


@pytest.mark.parametrize("rotary", [32, 20])
def test_append_to_a_cache_past_32_bits(B, rotary):
    """Rows past 2^29, codes past 2^33 bytes, in every kind of append."""
    for mode, interleaved in ((2, False), (2, True), (1, False)):
        dim, kv, page, pages = 64 if mode == 1 else 32, 8, 128, 600000
        cache = B.kv_cache_empty(pages, kv, page, dim, mode)
        small = B.kv_cache_empty(1, kv, page, dim, mode)
        table = B.rope_table(100, rotary, interleaved=interleaved)
        k, v = (synth.bf16_normal((page, kv, dim), 1.0, seed=s).cuda() for s in (1, 2))
        slots, pos = torch.arange(page, device="cuda"), torch.arange(page, dtype=torch.int32, device="cuda") % 100
        B.kv_append_rope(cache, table, k, v, slots + (pages - 1) * page, pos)
        B.kv_append_rope(small, table, k, v, slots, pos)
        assert all(torch.equal(a[-1], b[0]) for a, b in zip(cache.tensors[:4], small.tensors[:4]))
        assert not any(bool(t[:-1:5000].any()) for t in cache.tensors[:4])
        del cache


@pytest.mark.parametrize("interleaved", [False, True])
def test_one_token_of_heads_before_tokens(B, interleaved):
    """A single token of a [heads, tokens, head_dim] buffer whose heads lie more than 2^31 / 64 elements apart: rotated from there, in
    place, and appended."""
    heads, tokens, dim, at = 64, 300000, 128, 299998
    buffer = torch.zeros((heads, tokens, dim), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    x = synth.bf16_normal((2, heads, dim), 1.0, seed=7).cuda()
    buffer[at:at + 2] = x
    table, pos = B.rope_table(300, dim, interleaved=interleaved), ints([250, 251])
    want = B.rope(table, x, pos)
    assert torch.equal(B.rope(table, buffer[at + 1:], pos[1:]), want[1:])
    a, b = (B.kv_cache_empty(1, heads, 16, dim) for _ in range(2))
    slots = torch.arange(2, device="cuda")
    B.kv_append_rope(a, table, x, x, slots, pos)
    for i in range(2):
        one = buffer[at + i:at + i + 1]
        assert torch.equal(B.kv_append_rope(b, table, one, one, slots[i:i + 1], pos[i:i + 1], q=one), want[i:i + 1])
    assert all(torch.equal(s, t) for s, t in zip(a.tensors[:4], b.tensors[:4]))
    one = buffer[at + 1:]
    assert B.rope(table, one, pos[1:], out=one) is one and torch.equal(one, want[1:]) and torch.equal(buffer[at:at + 1], x[:1])
    assert not buffer[:at].any()
