"""rms_norm against 64 bits: sums and bf16 results within their rounding, codes and scales within what fp32's last bits
may make of them (see layer_reference.check_codes)."""
import numpy as np
import pytest
import torch

import layer_reference as R
import oracle
from block_scaled_fp4_fp_gb300 import synth
from helpers import u8, u32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.fp4_init(0)
    return binding


def inputs(rows, cols, seed=0, std=1.0):
    x, r = synth.bf16_normal((rows, cols), std, seed=seed), synth.bf16_normal((rows, cols), 3 * std, seed=seed + 1)
    w = (1 + 0.3 * synth.bf16_normal((1, cols), 1.0, seed=seed + 2).float()).bfloat16().view(-1)
    x[:, :: max(1, cols // 3)] *= 16
    return x, r, w


# y's error before its rounding: h, rstd (2^-24 and its own argument's error, which is below that), two products
Y = 4 * 2.0 ** -24


def check(B, x, r, w, eps, got, mode=None, gs=None, tiled=False):
    h, y = R.rms_norm(x, w, eps, r)
    if r is not None:
        R.assert_within(got.sum, h, 2.0 ** -24 * np.abs(h), "sum")
    if got.out is not None:
        R.assert_within(got.out, y, Y * np.abs(y), "out")
    if mode is not None:
        scales = u8(got.scales)
        if tiled:
            linear = np.empty((x.shape[0], x.shape[1] // R.GROUP[mode]), np.uint8)
            rr, cc = np.indices(linear.shape)
            pc = (linear.shape[1] + 3) // 4 * 4
            at = ((rr // 128) * (pc // 4) + cc // 4) * 512 + (rr % 32) * 16 + ((rr % 128) // 32) * 4 + cc % 4
            linear = scales.reshape(-1)[at]
            assert np.array_equal(oracle.tile_scales(linear), scales)  # and the padding is zero
            scales = linear
        R.check_codes(u32(got.xq), scales, y, Y * np.abs(y), mode, np.float64(np.float32(1.0 if gs is None else gs)))


SHAPES = [(1, 8), (1, 5120), (2, 16), (3, 2880), (129, 128), (7, 17408), (2, 32768), (1000, 64), (5, 24), (33, 264), (65, 8200),
          (4, 1024), (300, 520), (31, 16408)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_bf16(B, rows, cols, residual):
    x, r, w = inputs(rows, cols, seed=cols)
    r = r if residual else None
    got = B.rms_norm(x.cuda(), w.cuda(), residual=None if r is None else r.cuda())
    assert got.xq is None and got.scales is None and (got.sum is None) == (r is None)
    check(B, x, r, w, 1e-6, got)
    got = B.rms_norm(x.cuda(), None, eps=0.5, residual=None if r is None else r.cuda())
    check(B, x, r, None, 0.5, got)


FP4 = [(1, 5120), (3, 2880), (129, 128), (7, 17408), (2, 32768), (1000, 64), (1, 32), (37, 96), (257, 1056), (130, 224), (5, 8224)]


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rows,cols", FP4)
def test_four_bits(B, rows, cols, mode, layout):
    x, r, w = inputs(rows, cols, seed=cols + mode)
    gs = 0.0071 if mode == 2 and rows != 3 else None
    dgs = None if gs is None else torch.tensor(gs, device="cuda")
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda") if rows % 2 else None
    got = B.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), mode=mode, global_scale=dgs, layout=layout, out=out)
    check(B, x, r, w, 1e-6, got, mode, gs, layout == 1)
    # the same bits without residual and weight as with a residual of zeros and a weight of ones
    a = B.rms_norm(x.cuda(), mode=mode, global_scale=dgs, layout=layout)
    b = B.rms_norm(x.cuda(), torch.ones_like(w).cuda(), residual=torch.zeros_like(r).cuda(), mode=mode, global_scale=dgs, layout=layout)
    assert torch.equal(a.xq, b.xq) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("cols", [16, 48, 80, 112, 272])
@pytest.mark.parametrize("layout", [0, 1])
def test_scale_columns_that_are_no_whole_words(B, cols, layout):
    x, r, w = inputs(67, cols, seed=cols)
    check(B, x, None, w, 1e-6, B.rms_norm(x.cuda(), w.cuda(), mode=2, layout=layout), 2, None, layout == 1)
    # scales at an odd address
    n = np.prod(B.scales_shape(67, cols, 16, layout))
    buf = torch.full((n + 3,), 77, dtype=torch.uint8, device="cuda")
    sc = buf[1:1 + n].view(B.scales_shape(67, cols, 16, layout))
    check(B, x, None, w, 1e-6, B.rms_norm(x.cuda(), w.cuda(), mode=2, layout=layout, scales=sc), 2, None, layout == 1)
    assert buf[0] == 77 and (buf[1 + n:] == 77).all()


def test_codes_of_representable_results_are_the_quantizers(B):
    """Rows whose result is a bf16 number: what fp4_quantize makes of it, bit for bit."""
    g = torch.Generator().manual_seed(3)
    x = torch.where(torch.rand((64, 512), generator=g) < 0.5, -1.0, 1.0).bfloat16()  # rms 1, eps 0: y is the weight, signed
    w = synth.bf16_normal((1, 512), 1.0, seed=9).view(-1)
    for mode in (2, 1):
        got = B.rms_norm(x.cuda(), w.cuda(), eps=0.0, mode=mode, layout=1)
        xq, sc = B.fp4_quantize((x.float() * w.float()).bfloat16().cuda(), mode, layout=1)
        assert torch.equal(got.xq, xq) and torch.equal(got.scales, sc)


def test_views_and_in_place(B):
    """Rows of wider matrices; the sum written over the residual, or over x; the result over x.  Nothing beside them changes."""
    rows, cols = 77, 1280
    x, r, w = inputs(rows, cols, seed=4)
    wide = torch.full((rows + 1, 2 * cols + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    xv, rv = wide[:rows, :cols], wide[:rows, cols + 8:2 * cols + 8]
    xv.copy_(x)
    rv.copy_(r)
    want = B.rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
    check(B, x, r, w, 1e-6, want)
    got = B.rms_norm(xv, w.cuda(), residual=rv, sum_out=rv)
    assert got.sum is rv and torch.equal(rv, want.sum) and torch.equal(got.out, want.out) and torch.equal(xv.cpu(), x)
    rest = torch.ones_like(wide, dtype=torch.bool)
    rest[:rows, :cols] = False
    rest[:rows, cols + 8:2 * cols + 8] = False
    assert (wide[rest] == 7.0).all()
    rv.copy_(r)
    B.rms_norm(xv, w.cuda(), residual=rv, sum_out=xv)
    assert torch.equal(xv, want.sum) and torch.equal(rv.cpu(), r)
    xc = x.cuda()
    assert torch.equal(B.rms_norm(xc, w.cuda(), residual=r.cuda(), out=xc).out, want.out) and torch.equal(xc, want.out)
    one = wide[:1, 8:cols + 8]  # a single row, whatever its stride says
    assert B.rms_norm(one.as_strided((1, cols), (8, 1)), w.cuda()).out.shape == (1, cols)


@pytest.mark.parametrize("cols", [64, 5120, 9000])
def test_the_whole_range(B, cols):
    """Squares that fp32 does not hold, rows of zeros, and eps where it counts."""
    rows = 10
    x = synth.bf16_normal((rows, cols), 1.0, seed=cols)
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3] *= 1e-38  # mostly subnormal
    x[4] *= 1e19
    x[5] *= 1e-13
    x[6, :] = 0
    x[6, 5] = 3e38
    x[7] *= 1e-20
    w = synth.bf16_normal((1, cols), 1.0, seed=1).view(-1)
    for eps in (0.0, 1e-30, 1e-12, 1e-6):
        eps = float(np.float32(eps))
        got = B.rms_norm(x.cuda(), w.cuda(), eps=eps)
        check(B, x, None, w, eps, got)
        assert (got.out[2] == 0).all()
    if cols % 32:  # (no MXFP4 row)
        return
    zero = B.rms_norm(x[2:3].cuda(), w.cuda(), eps=0.0, mode=1)
    assert not (zero.xq.cpu().numpy().view(np.uint32) & 0x77777777).any() and not zero.scales.any()


def test_infinities_and_nans_stay_in_their_rows(B):
    for cols in (64, 2048):
        x = synth.bf16_normal((6, cols), 1.0, seed=2)
        x[1, 3] = float("inf")
        x[4, 7] = float("nan")
        out = B.rms_norm(x.cuda()).out.cpu()
        assert out[1, 3].isnan() and (out[1, :3] == 0).all() and (out[1, 4:] == 0).all() and out[4].isnan().all()
        clean = [0, 2, 3, 5]
        assert torch.equal(out[clean], B.rms_norm(x[clean].cuda()).out.cpu())


def test_on_a_stream_and_from_a_graph(B):
    x, r, w = inputs(50, 2880, seed=6)
    want = B.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), mode=2, layout=1)
    s = torch.cuda.Stream()
    xd, rd, wd = torch.zeros_like(x).cuda(), torch.zeros_like(r).cuda(), w.cuda()
    torch.cuda.synchronize()
    got = B.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), mode=2, layout=1, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.rms_norm(xd, wd, residual=rd, mode=2, layout=1)
        again = B.rms_norm(got.sum, wd, mode=2, layout=1)
    xd.copy_(x)
    rd.copy_(r)
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    twice = B.rms_norm(want.sum, wd, mode=2, layout=1)
    assert torch.equal(again.xq, twice.xq) and torch.equal(again.scales, twice.scales)


def test_many_rows(B):
    """More rows than a grid's other axes hold, sampled."""
    rows, cols = 150001, 64
    x = synth.bf16_normal((rows, cols), 1.0, seed=8)
    got = B.rms_norm(x.cuda(), mode=1, layout=1)
    pick = np.r_[0:50, 65530:65600, rows - 50:rows]
    part = B.rms_norm(x[pick].cuda(), mode=1)
    assert torch.equal(got.xq.cpu()[pick], part.xq.cpu())
    assert got.scales.shape == B.scales_shape(rows, cols, 32, 1)


def test_elements_past_32_bits(B):
    """Rows whose elements lie past 2^31 (and their bytes past 2^32): the same bits as on their own."""
    rows, cols = 140000, 16384
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    pick = torch.tensor([0, 65535, 131071, 131073, rows - 1])
    part = synth.bf16_normal((len(pick), cols), 1.0, seed=3).cuda()
    x.zero_()
    x[pick.cuda()] = part
    got = B.rms_norm(x, residual=x, mode=2, layout=1, sum_out=x)
    want = B.rms_norm(part, residual=part, mode=2)
    assert torch.equal(x[pick.cuda()], want.sum) and torch.equal(got.xq[pick.cuda()], want.xq)
    r, c = pick[:, None].cuda(), torch.arange(cols // 16, device="cuda")[None]
    at = ((r // 128) * (cols // 64) + c // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + c % 4
    assert torch.equal(got.scales.view(-1)[at], want.scales)
    assert int((got.xq != 0).any(-1).sum()) == len(pick)


def massive(rows, cols, channels, seed):
    """Normal rows with channels that hold nearly all of a row's squares, as a residual stream has them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    for c in channels:
        x[:, c] = 3000 * (1 + 0.01 * x[:, c])
    return x.bfloat16()


# 1/rms of such rows before what is made of it: its rounding (2^-24), the square root's own arithmetic and the sum of squares.  The
# other channels hold at most 2^-8 of the sum and their chains lose at most 17 times 2^-24 of that, 2^-28; the rest is exact.
RSTD = 2.0 ** -24 + 2.0 ** -27


@pytest.mark.parametrize("rows,cols,channels", [(4096, 5120, [5]), (4096, 5120, [5, 4000]), (200, 5120, [3777]), (1200, 17408, [17000]), (8000, 2880, [0]),
                                                (30000, 512, [100]), (60000, 128, [5, 9]), (3000, 1024, [1023]), (3000, 64, [33]), (1, 5120, [9]), (50000, 24, [17])])
def test_massive_channels(B, rows, cols, channels):
    """Each result is the rounding of a value within 1/rms's and one product's error of the exact one."""
    x = massive(rows, cols, channels, cols)
    out = B.rms_norm(x, eps=float(np.float32(1e-6))).out.double()
    h = x.double()
    y = h / (h.square().mean(-1, keepdim=True) + float(np.float32(1e-6))).sqrt()
    b = RSTD + 2.0 ** -24
    half = torch.ldexp(torch.ones_like(out), torch.frexp(out.abs().clamp(min=2.0 ** -120)).exponent - 9)  # half a step of bf16
    off = (out - y).abs() - half - b * y.abs()
    assert off.max() <= 0, f"{int((off > 0).sum())} elements, by up to {float((off / y.abs()).max()) * 2 ** 24:.2f} of 2^-24"


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("rows,cols,channels", [(300, 5120, [5, 4000]), (1000, 128, [9]), (2, 17408, [3000]), (700, 2880, [2879])])
def test_massive_channels_in_four_bits(B, rows, cols, channels, mode):
    x, r = massive(rows, cols, channels, 1).cpu(), synth.bf16_normal((rows, cols), 1.0, seed=2)
    w = (1 + 0.3 * synth.bf16_normal((1, cols), 1.0, seed=3).float()).bfloat16().view(-1)
    gs = float(np.float32(0.0003)) if mode == 2 else None  # (the other channels' results are near 0.02)
    got = B.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), mode=mode, global_scale=None if gs is None else torch.tensor(gs, device="cuda"))
    y = R.rms_norm(x, w, float(np.float32(1e-6)), r)[1]
    R.check_codes(u32(got.xq), u8(got.scales), y, (RSTD + 3 * 2.0 ** -24) * np.abs(y), mode, 1.0 if gs is None else gs)


@pytest.mark.parametrize("cols", [128, 512])
def test_a_rows_bits_do_not_depend_on_its_neighbours(B, cols):
    """Rows that share a warp with massive ones: the same bits as among others."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn((400000, cols), generator=g, device="cuda").bfloat16()
    beside = x.clone()
    beside[::8, 5] = 3000
    a, b = B.rms_norm(x).out, B.rms_norm(beside).out
    rest = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
    rest[::8] = False
    assert int((a[rest] != b[rest]).sum()) == 0
