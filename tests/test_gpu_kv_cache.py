"""kv_plan and kv_append against plain implementations: the plan token by token on
the host, the append bit for bit against the oracle's quantizer."""
import numpy as np
import pytest
import torch

import kv_reference as R
from block_scaled_fp4_fp_gb300 import synth
from helpers import u32, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.fp4_init(0)
    return binding


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def lengths(case):
    g = np.random.RandomState(len(case))
    return {
        "one request, first token": ([0], [1]),
        "one long prompt": ([0], [5000]),
        "decode": (list(g.randint(0, 300, 64)), [1] * 64),
        "page borders": ([0, 15, 16, 17, 63, 64, 65, 127, 128], [1, 1, 1, 0, 1, 1, 64, 2, 128]),
        "idle requests": ([0, 0, 7, 0, 40], [0, 0, 0, 0, 0]),
        "idle at both ends": ([9, 0, 3, 130, 0], [0, 0, 5, 17, 0]),
        "mixed 1300": (list(g.randint(0, 700, 1300)), list(g.randint(0, 40, 1300) * (g.rand(1300) < 0.6))),
    }[case]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("pad", [0, 37])
@pytest.mark.parametrize("case", ["one request, first token", "one long prompt", "decode", "page borders",
                                  "idle requests", "idle at both ends", "mixed 1300"])
def test_plan_matches_the_host(B, case, page, pad):
    cached, new = ([int(x) for x in v] for v in lengths(case))
    tokens = max(1, sum(new) + pad)
    total_pages = sum(-(-(c + n) // page) for c, n in zip(cached, new))
    g = np.random.RandomState(page + pad)
    ids = g.permutation(total_pages + 5).astype(np.int32)
    maxp = max(-(-(c + n) // page) for c, n in zip(cached, new)) + 2
    table = np.full((len(cached), maxp + 3), -7, np.int32)  # a row pitch past max_pages, entries marked
    at = 0
    for b, c in enumerate(cached):
        k = -(-c // page)
        table[b, :k] = ids[at:at + k]
        at += k
    free = ids[at:]
    want = R.plan(cached, new, free, table, page, tokens)
    dt = torch.from_numpy(table).cuda()
    got = B.kv_plan(ints(cached), ints(new), torch.from_numpy(free).cuda(), dt[:, :maxp], page, tokens)
    assert B.fp4_check_device_error() == B.FP4_OK
    assert np.array_equal(dt.cpu().numpy(), want[0])
    assert np.array_equal(got.total_lens.cpu().numpy(), want[1])
    assert np.array_equal(got.query_start.cpu().numpy(), want[2])
    assert np.array_equal(got.slot_map.cpu().numpy(), want[3])
    assert np.array_equal(got.positions.cpu().numpy(), want[4])
    assert int(got.pages_taken) == want[5]


def test_plan_reports_what_does_not_fit(B):
    """Too few free pages, a full table row, too small a token buffer: reported, and nothing outside is written."""
    def go(cached, new, nfree, maxp, tokens):
        table = torch.full((len(cached), maxp + 1), -7, dtype=torch.int32, device="cuda")
        table[:, 0] = torch.arange(len(cached))
        free = torch.arange(100, 100 + nfree, dtype=torch.int32, device="cuda")
        buf = torch.full((tokens + 8,), -99, dtype=torch.int64, device="cuda")
        B_ = len(cached)
        pl = B.KvPlan(torch.empty(B_, dtype=torch.int32, device="cuda"),
                      torch.empty(B_ + 1, dtype=torch.int32, device="cuda"), buf[:tokens],
                      torch.empty(tokens, dtype=torch.int32, device="cuda"),
                      torch.zeros((), dtype=torch.int32, device="cuda"))
        B.kv_plan(ints(cached), ints(new), free, table[:, :maxp], 16, tokens, plan=pl)
        st = B.fp4_check_device_error()
        assert (buf[tokens:] == -99).all() and (table[:, maxp:] == -7).all()
        return st, buf[:tokens].tolist(), table[:, :maxp].tolist()

    st, slots, _ = go([16, 16], [16, 16], 1, 4, 32)  # one page for two requests that need one each
    assert st == B.FP4_ERR_INVALID_ARG
    assert slots[:16] == list(range(1600, 1616)) and slots[16:] == [-1] * 16
    st, slots, table = go([16], [40], 8, 2, 40)  # the row holds two pages, three are needed
    assert st == B.FP4_ERR_INVALID_ARG
    assert slots[:16] == list(range(1600, 1616)) and slots[16:] == [-1] * 24 and table == [[0, 100]]
    st, slots, _ = go([0], [20], 8, 2, 16)
    assert st == B.FP4_ERR_INVALID_ARG and slots == list(range(1600, 1616))
    st, slots, _ = go([-5], [3], 8, 2, 3)
    assert st == B.FP4_ERR_INVALID_ARG and slots == [1600, 1601, 1602]
    st, slots, _ = go([4], [3], 0, 2, 3)  # fits the page it has: no free page needed
    assert st == B.FP4_OK and slots == [4, 5, 6]


@pytest.mark.parametrize("mode", [2, 1])
@pytest.mark.parametrize("dim,heads,tokens,page", [(128, 8, 77, 64), (64, 1, 1, 16), (128, 40, 1, 128), (32, 3, 65, 32),
                                                   (256, 2, 130, 16), (96, 5, 33, 32)])
@pytest.mark.parametrize("gs", [False, True])
def test_append_matches_the_oracle(B, mode, dim, heads, tokens, page, gs):
    if gs and mode == 1:
        pytest.skip("MXFP4 has no global scale")
    pages = tokens // page + 3
    rng = np.random.RandomState(tokens)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 3:
        slots[2] = -1  # a padding token
    # k and v lie in one row with other heads, as the fused projection leaves them
    qkv = synth.bf16_normal((tokens, 3 + 2 * heads, dim), 1.0, seed=dim + tokens)
    qkv[0, 3] = 0  # an all-zero head: scale byte 0
    if tokens > 1:
        qkv[1] *= 1e4
    k, v = qkv[:, 3:3 + heads], qkv[:, 3 + heads:]
    g = [torch.tensor(float(t.abs().max()) / 2688, dtype=torch.float32) if gs else None for t in (k, v)]
    words, groups = dim // 8, dim // B.GROUP[mode]
    old = [np.random.RandomState(5).randint(-2 ** 31, 2 ** 31, (pages, heads, page, words)).astype(np.int32),
           np.random.RandomState(6).randint(0, 256, (pages, heads, page, groups)).astype(np.uint8)]
    t = [torch.from_numpy(a.copy()).cuda() for a in (old[0], old[1], old[0], old[1])]
    cache = B.kv_cache(*t, mode, *[None if x is None else x.cuda() for x in g])
    d = qkv.cuda()
    B.kv_append(cache, d[:, 3:3 + heads], d[:, 3 + heads:], torch.from_numpy(slots).cuda())
    assert B.fp4_check_device_error() == B.FP4_OK
    for x, gx, codes, scales in ((k, g[0], t[0], t[1]), (v, g[1], t[2], t[3])):
        c, s = R.quantize(x.reshape(-1, dim).contiguous(), mode, None if gx is None else gx.item())
        wc, ws = old[0].view(np.uint32).copy(), old[1].copy()
        for i, slot in enumerate(slots):
            if slot >= 0:
                wc[slot // page, :, slot % page] = c.reshape(tokens, heads, words)[i]
                ws[slot // page, :, slot % page] = s.reshape(tokens, heads, groups)[i]
        assert np.array_equal(u32(codes), wc) and np.array_equal(u8(scales), ws)


def test_append_skips_and_reports_a_slot_past_the_cache(B):
    cache = B.kv_cache_empty(2, 1, 16, 64)
    k = synth.bf16_normal((3, 1, 64), 1.0, seed=1).cuda()
    B.kv_append(cache, k, k, torch.tensor([0, 32, 31], device="cuda"))
    assert B.fp4_check_device_error() == B.FP4_ERR_INVALID_ARG
    codes = cache.tensors[0]
    assert codes[0, 0, 0].any() and codes[1, 0, 15].any() and int((codes != 0).any(-1).sum()) == 2


def test_the_cache_reads_as_matrices_of_the_library(B):
    """What kv_append stored, fp4_dequantize reads: one row per (page, head, slot)."""
    cache = B.kv_cache_empty(4, 2, 32, 128, B.MODE_MXFP4)
    k = synth.bf16_normal((100, 2, 128), 1.0, seed=2).cuda()
    B.kv_append(cache, k, -k, torch.arange(100, device="cuda"))
    kc, ks, vc, vs = cache.tensors[:4]
    dk = B.fp4_dequantize(kc.view(-1, 16), ks.view(-1, 4), mode=B.MODE_MXFP4).view(4, 2, 32, 128)
    dv = B.fp4_dequantize(vc.view(-1, 16), vs.view(-1, 4), mode=B.MODE_MXFP4).view(4, 2, 32, 128)
    got = dk.transpose(1, 2).reshape(128, 2, 128)[:100]
    xq, xs = B.fp4_quantize(k.reshape(-1, 128), B.MODE_MXFP4)
    assert torch.equal(got.reshape(-1, 128), B.fp4_dequantize(xq, xs, mode=B.MODE_MXFP4))
    assert torch.equal(dk, -dv)


def test_plan_takes_no_page_that_no_row_holds(B):
    """Where a table row is full, the pages it has no entry for stay free: the next request's are the next of the list, and
    pages_taken counts what the rows hold."""
    table = torch.full((4, 3), -7, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(4)
    free = torch.arange(100, 109, dtype=torch.int32, device="cuda")
    # one page too many by three; exactly full; past its row already; one that fits
    pl = B.kv_plan(ints([16, 16, 100, 16]), ints([80, 32, 30, 16]), free, table, 16, 158)
    assert B.fp4_check_device_error() == B.FP4_ERR_INVALID_ARG
    assert table.tolist() == [[0, 100, 101], [1, 102, 103], [2, -7, -7], [3, 104, -7]]
    assert int(pl.pages_taken) == 5
    slots = pl.slot_map.tolist()
    assert slots[:32] == list(range(1600, 1632)) and slots[32:80] == [-1] * 48
    assert slots[80:112] == list(range(1632, 1664)) and slots[112:142] == [-1] * 30
    assert slots[142:] == list(range(1664, 1680))
