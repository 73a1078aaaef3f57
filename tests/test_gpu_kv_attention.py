"""kv_attention against a 64-bit implementation over the decoded cache.

Tolerance, element by element, with A = sum_j p_j |v_j| / sum_j p_j:
    |out - exact| <= 2^-8 |exact| + ((1 + 2^-8) exp(2 ds) - 1) A + 2^-126
The first term is the bf16 rounding of the result (2^-9) with room for the
division; a kernel may hold p in as few as 8 significant bits (2^-9 of every
p, and of their sum), which moves the result by at most 2^-8 A; and scores may be
off by ds = 2^-16 max|q| max_j |k_j|_1 scale: the tensor-core form writes q as
terms that leave 2^-17 of the row's largest element, and fp32 sums add less than as
much again.  A shift of ds moves every p by a factor within exp(+-ds), the
quotient by at most exp(2 ds).  Below 2^-126 bf16 has no normal numbers."""
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


def check(B, p, scale=None, lse=True, ws=None, q=None):
    cache, t = p.cuda(B)
    if q is not None:
        t["q"] = q
    mq = max(1, max(p.new))
    if ws is None:
        ws = B.kv_attention_workspace(cache, len(p.new), p.q_heads, mq)
    out = torch.full((p.q.shape[0], p.q_heads, p.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    sums = torch.full((p.q.shape[0], p.q_heads), 7.0, device="cuda") if lse else None
    B.kv_attention(cache, t["q"], t["query_start"], t["total_lens"], t["block_table"], ws, max_query_len=mq,
                   scale=scale, window=p.window, out=out, lse=sums)
    assert B.fp4_check_device_error() == B.FP4_OK
    want, wlse, bound = p.attention(scale)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"off by up to {np.abs(got - want).max():.3g}, {float((over > 0).mean()):.3g} over the bound"
    if lse:
        g = sums.double().cpu().numpy()
        empty = np.isneginf(wlse)
        assert np.isneginf(g[empty]).all()
        assert (np.abs(g - wlse)[~empty] <= p.lse_bound(scale)[~empty]).all()
    return out, ws


SHAPES = [  # dim, kv heads, group
    (128, 2, 8), (128, 3, 1), (128, 2, 5), (128, 1, 16), (128, 1, 33), (64, 2, 8), (64, 3, 1), (64, 1, 24),
    (256, 1, 8), (256, 2, 2), (256, 1, 16), (96, 2, 4), (32, 1, 2),
]


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,kv,group", SHAPES)
def test_decode(B, mode, dim, kv, group):
    """One token a request: contexts from one token, on both sides of pages, tiles and several tiles."""
    total = [1, 2, 15, 16, 17, 127, 128, 129, 255, 257, 700, 1300]
    p = R.Problem(mode, dim, kv, group, 64, [n - 1 for n in total], [1] * len(total), gs=mode == 2, seed=dim + group)
    check(B, p)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 300])
def test_decode_pages_and_windows(B, mode, page, window):
    total = [1, 90, 128, 200, 413, 1025]
    p = R.Problem(mode, 128, 2, 4, page, [n - 1 for n in total], [1] * len(total), window=window, seed=page + window)
    check(B, p)


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,kv,group", [(128, 2, 8), (128, 4, 1), (64, 1, 8), (64, 2, 3), (256, 1, 4), (32, 2, 2)])
@pytest.mark.parametrize("window", [0, 77])
def test_a_few_tokens(B, mode, dim, kv, group, window):
    """Ragged query counts, requests without queries among them, causal inside the step."""
    p = R.Problem(mode, dim, kv, group, 32, [0, 5, 126, 300, 0, 511, 40], [3, 4, 2, 0, 1, 4, 1], window=window, seed=dim)
    check(B, p)


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,kv,group", [(128, 2, 4), (128, 2, 1), (64, 2, 8), (64, 1, 5), (256, 1, 2), (96, 1, 2)])
@pytest.mark.parametrize("window", [0, 150])
def test_prompts(B, mode, dim, kv, group, window):
    """Whole prompts and chunks over what is cached; lengths around the tiles' edges."""
    p = R.Problem(mode, dim, kv, group, 16, [0, 130, 0, 300, 77, 0], [200, 129, 0, 64, 1, 257], window=window, gs=mode == 2,
                  seed=dim + window)
    check(B, p)


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("group", [1, 8])
def test_one_long_context(B, mode, group):
    """The work of one request is split along the context and joined."""
    p = R.Problem(mode, 128, 2, group, 128, [9000], [1], seed=group)
    check(B, p)


def test_sharp_and_rising_scores(B):
    """Scores that grow along the context (the running maximum moves in every tile) and that leave one key."""
    p = R.Problem(2, 128, 1, 8, 64, [1500, 640], [1, 1], seed=3, q_std=12.0)
    for b in range(2):  # later keys larger: scale bytes grow along the sequence
        j = np.arange(p.total[b])
        p.scales["k"][p.table[b, j // 64], 0, j % 64] = (0x20 + (24 * j // p.total[b]))[:, None].astype(np.uint8)
    check(B, p)
    check(B, p, scale=3.0)


def test_mxfp4_scales_far_apart(B):
    """V blocks whose scales differ by many powers of two between channels, and between tokens."""
    p = R.Problem(1, 128, 1, 8, 64, [700], [1], seed=4)
    p.scales["v"][:, :, :, 0] += 40
    p.scales["v"][:, :, :, 2] -= 60
    j = np.arange(701)
    p.scales["v"][p.table[0, j // 64], 0, j % 64] += (j % 7).astype(np.uint8)[:, None]
    p.scales["v"][p.unseen()] = 0xFF
    check(B, p)


def test_strided_queries_other_stream_and_reused_workspace(B):
    p = R.Problem(2, 128, 2, 8, 64, [3000, 10, 700], [1, 1, 1], gs=True, seed=8)
    wide = torch.zeros((3, p.q_heads + 5, p.dim), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + p.q_heads] = p.q.cuda()
    first, ws = check(B, p, q=wide[:, 2:2 + p.q_heads])
    again, _ = check(B, p, ws=ws)
    assert torch.equal(first, again)  # the same bits, the workspace left ready
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third, _ = check(B, p, ws=ws, lse=False)
    side.synchronize()
    assert torch.equal(first, third)


def test_captured_in_a_graph_with_new_lengths(B):
    """plan, append and attention captured once, replayed as the requests grow: lengths are read on the device."""
    batch, kv, heads, dim, page = 3, 2, 16, 128, 32
    cache = B.kv_cache_empty(40, kv, page, dim, B.MODE_NVFP4)
    lens = torch.tensor([0, 30, 63], dtype=torch.int32, device="cuda")
    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    table = torch.zeros((batch, 8), dtype=torch.int32, device="cuda")
    table[1, 0], table[2, 0], table[2, 1] = 1, 2, 3
    free = torch.arange(10, 40, dtype=torch.int32, device="cuda")
    qkv = torch.zeros((batch, heads + 2 * kv, dim), dtype=torch.bfloat16, device="cuda")
    ws = B.kv_attention_workspace(cache, batch, heads)

    def step():
        pl = B.kv_plan(lens, one, free, table, page, batch)
        B.kv_append(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], pl.slot_map)
        out = B.kv_attention(cache, qkv[:, :heads], pl.query_start, pl.total_lens, table, ws)
        lens.copy_(pl.total_lens)
        free.copy_(torch.roll(free, -1))
        return out

    g = torch.Generator(device="cuda").manual_seed(0)
    rows = [torch.randn(qkv.shape, generator=g, device="cuda").bfloat16() for _ in range(6)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    state = [t.clone() for t in (lens, table, free, *cache.tensors[:4])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for live in (False, True):
        for t, s in zip((lens, table, free, *cache.tensors[:4]), state):
            t.copy_(s)
        got = []
        for r in rows:
            qkv.copy_(r)
            if live:
                got.append(step().clone())
            else:
                graph.replay()
                got.append(out.clone())
        torch.cuda.synchronize()
        if live:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    assert B.fp4_check_device_error() == B.FP4_OK


def test_contract_violations_on_the_device_are_reported(B):
    for what in ("page id", "query length", "table row"):
        p = R.Problem(2, 128, 1, 8, 64, [200], [2], seed=1)
        cache, t = p.cuda(B)
        mq = 2
        if what == "page id":
            t["block_table"][0, 1] = p.num_pages
        elif what == "query length":
            mq = 1
        else:
            t["block_table"] = t["block_table"][:, :2]
        ws = B.kv_attention_workspace(cache, 1, p.q_heads, 2)
        B.kv_attention(cache, t["q"], t["query_start"], t["total_lens"], t["block_table"], ws, max_query_len=mq)
        assert B.fp4_check_device_error() == B.FP4_ERR_INVALID_ARG, what
        assert B.fp4_check_device_error() == B.FP4_OK


@pytest.mark.parametrize("mode,dim,kv,group", [(2, 128, 1, 4), (1, 64, 2, 4), (2, 64, 1, 9), (1, 128, 3, 1)])
@pytest.mark.parametrize("window", [0, 3000])
def test_chunks_over_long_contexts(B, mode, dim, kv, group, window):
    """Few rows in all, many keys: a request's keys are split over CTAs and joined, beside requests too short for that."""
    p = R.Problem(mode, dim, kv, group, 64, [6000, 0, 2500, 100], [40, 35, 3, 0], window=window, gs=mode == 2, seed=dim + kv)
    first, ws = check(B, p)
    again, _ = check(B, p, ws=ws)
    assert torch.equal(first, again)


@pytest.mark.parametrize("batch,kv", [(320, 2), (700, 1)])
def test_many_short_chunks(B, batch, kv):
    """More requests and heads than are dealt out in equal shares; more requests than a block has threads."""
    cached, new = [(7 * b) % 150 for b in range(batch)], [(b % 6) if b % 50 else 6 for b in range(batch)]
    p = R.Problem(1 + batch % 2, 64, kv, 8, 16, cached, new, seed=batch)
    check(B, p)


@pytest.mark.parametrize("dim", [64, 128])
def test_sharp_and_rising_scores_of_chunks(B, dim):
    """The rising scores of the decode test, for the kernel of many rows: its reference has to move."""
    p = R.Problem(2, dim, 1, 8, 64, [1500, 640], [9, 30], seed=3, q_std=12.0)
    for b in range(2):
        j = np.arange(p.total[b])
        p.scales["k"][p.table[b, j // 64], 0, j % 64] = (0x20 + (24 * j // p.total[b]))[:, None].astype(np.uint8)
    check(B, p)
    check(B, p, scale=3.0)


@pytest.mark.parametrize("new", [1, 12])
def test_a_workspace_serves_smaller_batches(B, new):
    full = R.Problem(2, 128, 2, 4, 64, [3000, 700, 10, 2000, 64], [new] * 5, seed=1)
    _, ws = check(B, full)
    for cached in ([4000], [5, 1000], [300, 2, 900]):
        check(B, R.Problem(2, 128, 2, 4, 64, cached, [new] * len(cached), seed=len(cached)), ws=ws)
        check(B, full, ws=ws)


@pytest.mark.parametrize("new", [1, 12])
@pytest.mark.parametrize("mode", [2, 1])
def test_timeout_injection_reports_and_recovers(B, mode, new):
    p = R.Problem(mode, 128, 2, 4, 64, [700, 90], [new] * 2, seed=1)
    cache, t = p.cuda(B)
    ws = B.kv_attention_workspace(cache, 2, p.q_heads, new)
    run = lambda: B.kv_attention(cache, t["q"], t["query_start"], t["total_lens"], t["block_table"], ws, max_query_len=new)
    first = run()
    B.fp4_debug_inject_wait_timeout(True)
    try:
        late = run()
        assert B.fp4_check_device_error() == B.FP4_ERR_TIMEOUT
        assert torch.equal(first, late)
    finally:
        B.fp4_debug_inject_wait_timeout(False)
    assert torch.equal(first, run())
    assert B.fp4_check_device_error() == B.FP4_OK


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim", [32, 96, 160, 192, 224])
@pytest.mark.parametrize("window", [0, 50])
def test_other_head_sizes(B, mode, dim, window):
    """Head sizes without a tensor-core form: one token, a few, a chunk, a request without queries."""
    p = R.Problem(mode, dim, 2, 3, 16, [0, 31, 257, 600, 12], [1, 3, 40, 1, 0], window=window, gs=mode == 2, seed=dim)
    check(B, p)


@pytest.mark.parametrize("mode,dim,kv,group", [(2, 128, 2, 4), (1, 64, 1, 8)])
@pytest.mark.parametrize("window", [0, 200])
def test_chunks_at_the_tiles_edges(B, mode, dim, kv, group, window):
    """127, 128, 129, 256 and 257 rows of a kv head in one call: items whose second tile has no rows, some, all; contexts of
    one, two and three key tiles."""
    rows = [127, 128, 129, 256, 257, 40]
    new = [-(-r // group) for r in rows]
    total = [130, 128, 300, 257, 129, 11]
    p = R.Problem(mode, dim, kv, group, 32, [max(t - n, 0) for t, n in zip(total, new)], new, window=window, gs=mode == 2, seed=kv + window)
    check(B, p)


@pytest.mark.parametrize("dim", [64, 128, 96])
@pytest.mark.parametrize("new", [1, 9])
def test_mxfp4_scales_at_the_ends_of_their_range(B, dim, new):
    """V blocks scaled by up to 2^119 and down to 2^-127, K blocks by 2^-127: any E8M0 scale counts for what it is."""
    p = R.Problem(1, dim, 1, 8, 16, [20 - new, 0], [new, new], seed=dim + new, q_std=0.05)
    g = np.random.RandomState(dim)
    p.scales["v"][:] = g.randint(236, 247, p.scales["v"].shape)
    p.scales["v"][..., -1] = g.randint(0, 4, p.scales["v"].shape[:-1])
    p.scales["k"][..., -1] = 0
    p.scales["v"][p.unseen()] = 0xFF
    p.scales["k"][p.unseen()] = 0xFF
    check(B, p)


@pytest.mark.parametrize("mode,dim,group", [(2, 128, 8), (1, 64, 4), (2, 256, 2)])
def test_calls_of_every_kind_take_turns_on_one_workspace(B, mode, dim, group):
    """Single tokens, a few, prompts, and the reverse, over contexts long enough that items are split: each call leaves the
    workspace ready for any other, whatever kernel and piece size it takes."""
    cases = {n: R.Problem(mode, dim, 2, group, 64, [12000] * 5, [n] * 5, seed=n) for n in (1, 2, 4, 12)}
    cache, _ = cases[12].cuda(B)
    ws = B.kv_attention_workspace(cache, 5, cases[12].q_heads, 12)
    for n in (4, 1, 12, 1, 4, 12, 2, 12, 4, 1):
        check(B, cases[n], ws=ws)
    small = R.Problem(mode, dim, 1, 2 * group, 64, [2500], [4], seed=9)  # other heads, another batch
    check(B, small, ws=ws)
    check(B, cases[1], ws=ws)


@pytest.mark.parametrize("dim", [64, 128, 96])
@pytest.mark.parametrize("new", [1, 12])
@pytest.mark.parametrize("window", [0, 40])
def test_a_negative_total_counts_as_no_keys(B, dim, new, window):
    """Down to the lowest 32-bit number, whose difference to a query count is no 32-bit number: zeros, and the others' results."""
    p = R.Problem(2, dim, 1, 8, 64, [300, 20, 700], [new] * 3, window=window, seed=dim + new)
    cache, t = p.cuda(B)
    ws = B.kv_attention_workspace(cache, 3, p.q_heads, new)
    call = lambda lse: B.kv_attention(cache, t["q"], t["query_start"], t["total_lens"], t["block_table"], ws, max_query_len=new,  # noqa: E731
                                      window=window, lse=lse)
    sums = torch.empty((3 * new, p.q_heads), device="cuda")
    want = call(None)
    for total in (-1, -2 ** 31 + 1, -2 ** 31):
        t["total_lens"][1] = total
        got = call(sums)
        assert B.fp4_check_device_error() == B.FP4_OK
        mine = slice(new, 2 * new)
        assert not got[mine].any() and torch.isneginf(sums[mine]).all()
        assert torch.equal(got[:new], want[:new]) and torch.equal(got[2 * new:], want[2 * new:])


@pytest.mark.parametrize("new", [1, 12])
def test_a_workspace_left_by_an_expired_wait_is_reported(B, new):
    """The mark of such a call: every later one reports it, until the workspace is zeroed."""
    p = R.Problem(2, 128, 2, 4, 64, [700, 90], [new] * 2, seed=1)
    cache, t = p.cuda(B)
    _, ws = check(B, p)
    run = lambda: B.kv_attention(cache, t["q"], t["query_start"], t["total_lens"], t["block_table"], ws, max_query_len=new)  # noqa: E731
    ws.view(torch.int32)[2] = 1
    for _ in range(2):
        run()
        assert B.fp4_check_device_error() == B.FP4_ERR_TIMEOUT
    ws.zero_()
    check(B, p, ws=ws)
    assert not ws.view(torch.int32)[:16].any()


def huge_values(B, dim, new):
    """4096 keys whose V is near bf16's largest numbers: their weighted mean is one of bf16's, their weighted sum is none of fp32's.
    All equal; of different sizes; under scores that rise by about 20 in log2 along the context."""
    for what in ("equal", "different", "rising"):
        p = R.Problem(1, dim, 1, 8, 64, [4096 - new, 70, 0], [new] * 3, seed=dim + new, q_std=0.3)
        g = np.random.RandomState(dim)
        if what == "equal":
            p.codes["v"][:], p.scales["v"][:] = 0x22222222, 127 + 120  # code 2 is 1
        else:
            p.scales["v"][:] = g.randint(240, 252, p.scales["v"].shape)
        if what == "rising":
            j = np.arange(4096)
            p.codes["k"][p.table[0, j // 64], 0, j % 64, 0] = 0x00000007  # channel 0 is 6 times a scale that grows
            p.scales["k"][p.table[0, j // 64], 0, j % 64, 0] = 120 + (7 * j // 4096)
            p.q[..., 0] = 1.75 * (dim / 64) ** 0.5
        for w, bad in (("v", 0xFF), ("k", 0xFF)):
            p.scales[w][p.unseen()] = bad
        check(B, p)


@pytest.mark.parametrize("dim,new", [(96, 1), (96, 9), (32, 1), (128, 1), (64, 2)])
def test_values_near_the_largest_numbers(B, dim, new):
    huge_values(B, dim, new)


@pytest.mark.parametrize("dim,new", [(64, 12), (128, 9), (128, 20), (64, 130)])
def test_values_near_the_largest_numbers_in_prompts(B, dim, new):
    huge_values(B, dim, new)


def test_values_near_the_largest_numbers_in_many_short_chunks(B):
    """Items handed out one by one, of which most have to be done again; twice, on one workspace."""
    batch = 320
    cached, new = [60 + (7 * b) % 150 for b in range(batch)], [(b % 6) if b % 50 else 6 for b in range(batch)]
    p = R.Problem(1, 64, 2, 8, 16, cached, new, seed=5, q_std=0.3)
    p.scales["v"][:] = np.random.RandomState(1).randint(236, 252, p.scales["v"].shape)
    p.scales["v"][p.unseen()] = 0xFF
    first, ws = check(B, p)
    again, _ = check(B, p, ws=ws)
    assert torch.equal(first, again)
