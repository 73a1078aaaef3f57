"""The operators around a decoder layer's products on several streams at once, and one after the other without a wait
between: the same bits as on their own."""
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


def calls(B):
    """name -> a call on inputs of its own that returns its outputs."""
    x, r = (synth.bf16_normal((700, 2880), 1.0, seed=s).cuda() for s in (1, 2))
    w = synth.bf16_normal((1, 2880), 1.0, seed=3).view(-1).cuda()
    g = torch.Generator().manual_seed(4)
    many, few = (torch.randint(-1, 32, (t, 4), generator=g, dtype=torch.int32).cuda() for t in (5000, 96))
    rope = B.rope_table(4000, 128)
    qkv = synth.bf16_normal((600, 12, 128), 1.0, seed=5).cuda()
    q, k, v = qkv.split([8, 2, 2], 1)
    slots, pos = torch.randperm(640, generator=g)[:600].cuda(), torch.arange(3000, 3600, dtype=torch.int32, device="cuda")
    plan = B.moe_sort(few, 32)
    y, weights = synth.bf16_normal((384, 2880), 1.0, seed=6).cuda(), torch.rand((96, 4), generator=g).cuda()

    def append():
        cache = B.kv_cache_empty(10, 2, 64, 128)
        return (B.kv_append_rope(cache, rope, k, v, slots, pos, q=q), *cache.tensors[:4])

    return {"norm": lambda: B.rms_norm(x, w, residual=r)[:2], "norm to 4 bits": lambda: B.rms_norm(x, w, residual=r, mode=2, layout=1)[1:],
            "sort, a cluster": lambda: B.moe_sort(many, 32), "sort, one CTA": lambda: B.moe_sort(few, 32),
            "rope": lambda: (B.rope(rope, q, pos),), "append": append, "combine": lambda: (B.moe_combine(y, plan.slot, weights),),
            "gradients": lambda: B.moe_combine_backward(x[:96], plan.slot, weights, y=y, offsets=plan.offsets)}


def test_at_once_and_in_a_row(B):
    todo = calls(B)
    want = {}
    for name, f in todo.items():
        want[name] = [t.clone() for t in f()]
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in todo]
    got = []
    torch.cuda.synchronize()
    for _ in range(20):
        for i, ((name, f), s) in enumerate(zip(todo.items(), streams)):
            with torch.cuda.stream(s):
                got.append((name, f()))
    for name, f in list(todo.items()) * 5:
        got.append((name, f()))
    torch.cuda.synchronize()
    for name, outs in got:
        assert len(outs) == len(want[name]) and all(torch.equal(a, b) for a, b in zip(outs, want[name])), name
    assert B.fp4_check_device_error() == B.FP4_OK


def test_graphs_of_one_call_share_nothing(B):
    """Two captured graphs of the same calls, replayed at once on two streams."""
    todo = calls(B)
    want = {name: [t.clone() for t in f()] for name, f in todo.items()}
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph, outs = torch.cuda.CUDAGraph(), {}
        with torch.cuda.graph(graph):
            for name, f in todo.items():
                outs[name] = f()
        graphs.append((graph, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, _, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, outs, _ in graphs:
        for name, o in outs.items():
            assert all(torch.equal(a, b) for a, b in zip(o, want[name])), name
