"""qmv right behind the quantizer that writes its weights, without a wait between: the same bits as with one.  (qmv streams its
first weights while the kernel before it drains.)"""
import pytest
import torch

from block_scaled_fp4_fp_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.fp4_init(0)
    return binding


def setup(B, N, K, mode):
    ws = [synth.bf16_normal((N, K), 0.02 * (i + 1), seed=i + N, device="cuda") for i in range(2)]
    gs = torch.tensor(2e-5, device="cuda") if mode == 2 else None
    x = synth.bf16_normal((K,), 1.0, seed=9, device="cuda")
    q, s = B.fp4_quantize(ws[0], mode, global_scale=gs)
    want = []
    for w in ws:
        B.fp4_quantize(w, mode, global_scale=gs, xq=q, scales=s)
        torch.cuda.synchronize()
        want.append(B.qmv(x, q, s, global_scale_w=gs, mode=mode))
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    return ws, gs, x, q, s, want


@pytest.mark.parametrize("N,K", [(34816, 5120), (5120, 5120), (5120, 17408), (1000, 512), (77, 160), (40000, 256)])
@pytest.mark.parametrize("mode", [2, 1])
def test_weights_that_were_just_quantized(B, N, K, mode):
    ws, gs, x, q, s, want = setup(B, N, K, mode)
    got = []
    for i in range(40):
        B.fp4_quantize(ws[i & 1], mode, global_scale=gs, xq=q, scales=s)
        got.append(B.qmv(x, q, s, global_scale_w=gs, mode=mode))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i & 1]) for i, y in enumerate(got))


@pytest.mark.parametrize("mode", [2, 1])
def test_codes_of_the_tiled_layout_with_linear_scales(B, mode):
    """The codes come from the second of two calls, whose scales are tiled."""
    ws, gs, x, q, s, want = setup(B, 17408, 5120, mode)
    st, spare = B.fp4_quantize(ws[0], mode, global_scale=gs, layout=B.SCALES_TILED)[1], torch.empty_like(q)
    got = []
    for i in range(40):
        B.fp4_quantize(ws[i & 1], mode, global_scale=gs, xq=spare, scales=s)
        B.fp4_quantize(ws[i & 1], mode, global_scale=gs, layout=B.SCALES_TILED, xq=q, scales=st)
        got.append(B.qmv(x, q, s, global_scale_w=gs, mode=mode))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i & 1]) for i, y in enumerate(got))


@pytest.mark.parametrize("mode", [2, 1])
def test_another_gemv_between(B, mode):
    """quantize, a GEMV over other weights (which releases the next launch at once), then the GEMV over what was quantized."""
    ws, gs, x, q, s, want = setup(B, 17408, 5120, mode)
    small = B.fp4_quantize(synth.bf16_normal((64, 5120), 0.02, seed=3, device="cuda"), mode, global_scale=gs)
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        B.fp4_quantize(ws[i & 1], mode, global_scale=gs, xq=q, scales=s)
        B.qmv(x, *small, global_scale_w=gs, mode=mode)
        got.append(B.qmv(x, q, s, global_scale_w=gs, mode=mode))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i & 1]) for i, y in enumerate(got))


@pytest.mark.parametrize("mode", [2, 1])
def test_in_a_graph(B, mode):
    ws, gs, x, q, s, want = setup(B, 17408, 5120, mode)
    graph, got = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for i in range(8):
            B.fp4_quantize(ws[i & 1], mode, global_scale=gs, xq=q, scales=s)
            got.append(B.qmv(x, q, s, global_scale_w=gs, mode=mode))
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i & 1]) for i, y in enumerate(got))
