"""moe_sort against a stable sort on the host, bit for bit; moe_combine and its gradients against 64 bits."""
import numpy as np
import pytest
import torch

import layer_reference as R
from block_scaled_fp4_fp_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.fp4_init(0)
    return binding


def routing(tokens, k, experts, seed=0, drop=0.0):
    """Skewed ids, the same expert twice among them."""
    g = np.random.RandomState(seed)
    ids = np.minimum((experts * g.rand(tokens, k) ** 2).astype(np.int32), experts - 1)
    ids[g.rand(tokens, k) < drop] = -1
    return ids


def check_sort(B, ids, experts, status=None):
    got = B.moe_sort(torch.from_numpy(ids).cuda(), experts)
    assert B.fp4_check_device_error() == (B.FP4_OK if status is None else status)
    for g, w, name in zip(got, R.moe_sort(ids, experts), got._fields):
        assert np.array_equal(g.cpu().numpy(), w), name
    return got


SORTS = [(1, 1, 1), (1, 8, 256), (3, 2, 7), (96, 4, 32), (31, 1, 1024), (33, 1, 2), (2048, 4, 32), (1024, 4, 60), (1025, 4, 60), (4097, 1, 1024),
         (5000, 8, 3), (40000, 6, 128), (2, 1024, 7), (300000, 1, 8), (70000, 8, 256)]


@pytest.mark.parametrize("tokens,k,experts", SORTS)
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort(B, tokens, k, experts, drop):
    check_sort(B, routing(tokens, k, experts, tokens + k, drop), experts)


@pytest.mark.parametrize("tokens", [5, 3000])
def test_sort_extremes(B, tokens):
    """All rows dropped; all to the last expert; the first half padding; extreme ids, reported where they are too large."""
    ids = np.full((tokens, 2), -1, np.int32)
    check_sort(B, ids, 16)
    check_sort(B, np.full_like(ids, 15), 16)
    half = routing(tokens, 2, 16)
    half[: tokens // 2] = -2 ** 31
    check_sort(B, half, 16)
    half[-1, 0] = 16
    check_sort(B, half, 16, B.FP4_ERR_INVALID_ARG)
    half[0, 0] = 2 ** 31 - 1
    check_sort(B, half, 16, B.FP4_ERR_INVALID_ARG)


def test_sort_from_a_graph_on_buffers_of_the_callers(B):
    """A captured sort, replayed on other ids; words beside the buffers stay."""
    i32 = torch.int32
    ids = torch.zeros((700, 4), dtype=i32, device="cuda")
    buf = torch.full((4, 2800 + 8), -9, dtype=i32, device="cuda")
    plan = B.MoeSort(buf[0, 4:2804], buf[1, 4:2804], buf[2, 4:2804].view(700, 4), buf[3, 4:4 + 33])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_sort(ids, 32, plan=plan)
    for seed in (1, 2):
        host = routing(700, 4, 32, seed, 0.1)
        ids.copy_(torch.from_numpy(host))
        graph.replay()
        for g, w in zip(plan, R.moe_sort(host, 32)):
            assert np.array_equal(g.cpu().numpy(), w)
    assert (buf[:, :4] == -9).all() and (buf[:3, 2804:] == -9).all() and (buf[3, 37:] == -9).all()


def combine_case(tokens, k, cols, experts=8, seed=0, drop=0.2):
    ids = routing(tokens, k, experts, seed, drop)
    slot = R.moe_sort(ids, experts)[2].astype(np.int32)
    y = synth.bf16_normal((tokens * k, cols), 1.0, seed=seed + 1)
    w = torch.softmax(synth.bf16_normal((tokens, k), 1.0, seed=seed + 2).float(), -1)
    r = synth.bf16_normal((tokens, cols), 2.0, seed=seed + 3)
    return slot, y, w, r


COMBINES = [(1, 1, 8), (1, 4, 5120), (96, 4, 5120), (7, 8, 2880), (33, 3, 1032), (5, 11, 264), (300, 2, 4104), (2, 40, 4160), (2000, 1, 16), (5003, 2, 512), (4870, 3, 1000)]


@pytest.mark.parametrize("tokens,k,cols", COMBINES)
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(B, tokens, k, cols, weights, residual):
    slot, y, w, r = combine_case(tokens, k, cols, seed=cols)
    valid = slot >= 0
    terms = np.where(valid[..., None], y.double().numpy()[np.maximum(slot, 0)], 0.0)
    if weights:
        terms = terms * w.double().numpy()[..., None]
    base = r.double().numpy() if residual else 0.0
    # k + 1 terms added in fp32: each partial sum, at most the sum of absolute values, is off by 2^-24 of itself
    most = (np.abs(terms).sum(1) + np.abs(base)) * (k * 2.0 ** -24)
    dev = lambda on, t: t.cuda() if on else None  # noqa: E731
    got = B.moe_combine(y.cuda(), torch.from_numpy(slot).cuda(), dev(weights, w), residual=dev(residual, r))
    assert B.fp4_check_device_error() == B.FP4_OK
    R.assert_within(got, base + terms.sum(1), most, "combine")
    if residual:
        rd = r.cuda()
        assert B.moe_combine(y.cuda(), torch.from_numpy(slot).cuda(), dev(weights, w), residual=rd, out=rd) is rd
        assert torch.equal(rd, got)


@pytest.mark.parametrize("tokens,k,cols", COMBINES)
@pytest.mark.parametrize("weights", [False, True])
def test_gradients(B, tokens, k, cols, weights):
    slot, y, w, _ = combine_case(tokens, k, cols, seed=cols + 1)
    kept = int((slot >= 0).sum())
    g = synth.bf16_normal((tokens, cols), 1.0, seed=4)
    gd, yd, wd = g.double().numpy(), y.double().numpy(), w.double().numpy() if weights else np.ones((tokens, k))
    dy, dw, size = np.zeros(y.shape), np.zeros((tokens, k)), np.zeros((tokens, k))
    for t in range(tokens):
        for j in range(k):
            if slot[t, j] >= 0:
                dy[slot[t, j]] = wd[t, j] * gd[t]
                dw[t, j] = gd[t] @ yd[slot[t, j]]
                size[t, j] = np.abs(gd[t]) @ np.abs(yd[slot[t, j]])
    s, offsets = torch.from_numpy(slot).cuda(), torch.tensor([0, kept], dtype=torch.int32, device="cuda")
    buf = torch.full_like(y, 3.0).cuda()
    a, b = B.moe_combine_backward(g.cuda(), s, w.cuda() if weights else None, y=y.cuda(), offsets=offsets, dy=buf)
    assert B.fp4_check_device_error() == B.FP4_OK and a is buf
    R.assert_within(a, dy, 2.0 ** -24 * np.abs(dy), "dy")
    # a product with each of a row's elements, added up in fp32 in any order: at most cols roundings of 2^-24 of the sum
    # of absolute values
    assert np.all(np.abs(b.cpu().double().numpy() - dw) <= cols * 2.0 ** -24 * size)
    assert (a[kept:] == 0).all() and (b.cpu().numpy()[slot < 0] == 0).all()
    # the same bits again; without y no weights' gradient; without offsets the rows of no slot stay
    c, d = B.moe_combine_backward(g.cuda(), s, w.cuda() if weights else None, y=y.cuda(), offsets=offsets)
    assert torch.equal(a, c) and torch.equal(b, d)
    buf = torch.full_like(y, 3.0).cuda()
    a, none = B.moe_combine_backward(g.cuda(), s, w.cuda() if weights else None, dy=buf)
    assert none is None and torch.equal(a[:kept], c[:kept]) and (a[kept:] == 3).all()


def test_gradients_against_differences(B):
    """moe_combine is linear in y and in the weights: differences of its fp32 sums (read through a residual that cancels
    them, so that bf16 shows the difference itself) against the gradients."""
    tokens, k, cols = 12, 3, 512
    slot, y, w, _ = combine_case(tokens, k, cols, seed=9, drop=0.1)
    s, g = torch.from_numpy(slot).cuda(), synth.bf16_normal((tokens, cols), 1.0, seed=10).cuda()
    yd, wd = y.cuda(), w.cuda()
    dy, dw = B.moe_combine_backward(g, s, wd, y=yd, offsets=torch.tensor([0, int((slot >= 0).sum())], dtype=torch.int32, device="cuda"))
    step = synth.bf16_normal(tuple(y.shape), 1.0, seed=11).cuda()
    left = (B.moe_combine(step, s, wd).double() * g.double())  # combine(y + step) - combine(y)
    right = step.double() * dy.double()
    assert abs(left.sum() - right.sum()) <= 2.0 ** -8 * 1.01 * (left.abs().sum() + right.abs().sum())
    dstep = synth.bf16_normal((tokens, k), 1.0, seed=12).float().cuda()
    left = B.moe_combine(yd, s, dstep).double() * g.double()  # combine(w + dstep) - combine(w)
    right = dstep.double() * dw.double()
    assert abs(left.sum() - right.sum()) <= 2.0 ** -8 * 1.01 * left.abs().sum() + 2.0 ** -20 * right.abs().sum()


def test_the_gathers_gradient(B):
    """gather_rows puts token t's row at each of its slots; its gradient adds them up again: moe_combine without weights."""
    ids = routing(200, 4, 16, 3, 0.1)
    plan = B.moe_sort(torch.from_numpy(ids).cuda(), 16)
    g = synth.bf16_normal((800, 256), 1.0, seed=1).cuda()
    got = B.moe_combine(g, plan.slot)
    want = torch.zeros((200, 256), dtype=torch.float64, device="cuda")
    kept = int(plan.offsets[-1])
    want.index_add_(0, plan.lhs_idx[:kept].long(), g[:kept].double())
    size = torch.zeros_like(want).index_add_(0, plan.lhs_idx[:kept].long(), g[:kept].double().abs())
    R.assert_within(got, want.cpu().numpy(), size.cpu().numpy() * 4 * 2.0 ** -24)


def test_slots_past_the_rows_are_reported(B):
    y, g = synth.bf16_normal((4, 64), 1.0, seed=1).cuda(), synth.bf16_normal((2, 64), 1.0, seed=2).cuda()
    slot = torch.tensor([[0, 4], [2 ** 31 - 1, 3]], dtype=torch.int32, device="cuda")
    out = B.moe_combine(y, slot)
    assert B.fp4_check_device_error() == B.FP4_ERR_INVALID_ARG
    assert torch.equal(out[0], y[0]) and torch.equal(out[1], y[3])
    dy, dw = B.moe_combine_backward(g, slot, y=y, dy=torch.zeros_like(y))
    assert B.fp4_check_device_error() == B.FP4_ERR_INVALID_ARG
    assert torch.equal(dy[0], g[0]) and torch.equal(dy[3], g[1]) and (dy[1:3] == 0).all()
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and dw[0, 0] != 0


def test_rows_that_are_not_read_may_hold_anything(B):
    """NaN in rows that no slot names reaches nothing."""
    y = synth.bf16_normal((6, 64), 1.0, seed=1).cuda()
    y[4:] = float("nan")
    slot = torch.tensor([[0, -1], [3, 2], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.full((3, 2), 0.5, device="cuda")
    w[0, 1] = w[2] = float("nan")  # nor the weights of dropped rows
    out = B.moe_combine(y, slot, w)
    assert out.isfinite().all() and (out[2] == 0).all()
    dy, dw = B.moe_combine_backward(torch.ones((3, 64), dtype=torch.bfloat16, device="cuda"), slot, w, y=y,
                                    offsets=torch.tensor([4], dtype=torch.int32, device="cuda"))
    assert dw.isfinite().all() and (dy[4:] == 0).all() and dy[[0, 2, 3]].isfinite().all()


def test_combine_from_a_graph(B):
    slot, y, w, r = combine_case(40, 4, 512, seed=2)
    s, yd, wd, rd = torch.from_numpy(slot).cuda(), y.cuda(), w.cuda(), r.cuda()
    want = B.moe_combine(yd, s, wd, residual=rd)
    graph = torch.cuda.CUDAGraph()
    out = rd.clone()
    with torch.cuda.graph(graph):
        B.moe_combine(yd, s, wd, residual=out, out=out)
    graph.replay()
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = B.moe_combine(yd, s, wd, residual=rd, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_elements_past_32_bits(B):
    """Rows of y past 2^31 elements, forward and back."""
    rows, cols, tokens = 300000, 8192, 6
    y = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([[0, rows - 1], [262143, 262145], [rows - 2, -1], [5, 6], [131072, 131073], [-1, -1]], dtype=torch.int32, device="cuda")
    live = slot[slot >= 0].long()
    y[live] = synth.bf16_normal((live.numel(), cols), 1.0, seed=6).cuda()
    g = synth.bf16_normal((tokens, cols), 1.0, seed=7).cuda()
    packed = torch.full_like(slot, -1)
    packed[slot >= 0] = torch.arange(live.numel(), dtype=torch.int32, device="cuda")
    assert torch.equal(B.moe_combine(y, slot), B.moe_combine(y[live], packed))
    dy, dw = B.moe_combine_backward(g, slot, y=y, dy=torch.zeros_like(y))
    want = B.moe_combine_backward(g, packed, y=y[live])
    assert torch.equal(dy[live], want[0]) and torch.equal(dw, want[1])
    assert int((dy != 0).any(-1).sum()) == live.numel()


@pytest.mark.parametrize("most", [1, 8, 9])
def test_sort_by_smaller_clusters(B, most):
    """The launches that a part of a GPU without room for 16 CTAs side by side gets: one tile and many a CTA, every id dropped,
    replayed from a graph, the same lists."""
    B.fp4_debug_limit_sort_ctas(most)
    try:
        for tokens, k, experts, drop in ((700, 3, 32, 0.0), (2049, 1, 1, 0.0), (4096, 4, 60, 0.3), (70000, 8, 256, 0.1), (9000, 8, 1024, 0.0), (3000, 2, 16, 1.0),
                                         (1, 1, 1, 0.0)):
            check_sort(B, routing(tokens, k, experts, tokens, drop), experts)
        ids = torch.zeros((9000, 4), dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan = B.moe_sort(ids, 64)
        host = routing(9000, 4, 64, 1, 0.2)
        ids.copy_(torch.from_numpy(host))
        graph.replay()
        for g, w in zip(plan, R.moe_sort(host, 64)):
            assert np.array_equal(g.cpu().numpy(), w)
    finally:
        B.fp4_debug_limit_sort_ctas(0)


def test_the_limit_of_a_sorts_cluster_is_checked(B):
    with pytest.raises(B.Fp4Error):
        B.fp4_debug_limit_sort_ctas(-1)
