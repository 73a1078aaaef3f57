"""Host-side checks of the paged-cache entry points (no GPU needed): bad calls are
refused before anything touches a device."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.lib()
    return binding


P = 256  # never dereferenced: every call below fails validation first


def cache(B, **kw):
    f = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, global_scale_k=None, global_scale_v=None, num_pages=4,
             page_size=64, kv_heads=2, head_dim=128, mode=B.MODE_NVFP4)
    f.update(kw)
    return B.KvCache(**f)


BAD_CACHES = [
    (dict(mode=0), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"), (dict(page_size=256), "UNSUPPORTED"),
    (dict(head_dim=80), "UNSUPPORTED"), (dict(head_dim=288), "UNSUPPORTED"), (dict(head_dim=0), "INVALID_ARG"),
    (dict(k_codes=None), "INVALID_ARG"), (dict(v_scales=None), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(kv_heads=0), "INVALID_ARG"), (dict(num_pages=1 << 24), "INVALID_ARG"),
    (dict(mode=1, global_scale_k=P), "INVALID_ARG"), (dict(v_codes=P + 8), "ALIGNMENT"),
    (dict(global_scale_v=P + 2), "ALIGNMENT"),
]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_bad_caches_are_refused(B, change, want):
    L, c = B.lib(), cache(B, **change)
    want = getattr(B, "FP4_ERR_" + want)
    assert L.kv_append(ctypes.byref(c), P, 512, 128, P, 512, 128, P, 4, None) == want
    assert L.kv_attention(ctypes.byref(c), P, 512, 128, 4, 4, P, P, 4, P, 8, 8, 1, 0.1, 0, P, 1 << 40, P, None,
                          None) == want
    assert L.kv_append(None, P, 512, 128, P, 512, 128, P, 4, None) == B.FP4_ERR_INVALID_ARG


def test_append_refusals(B):
    L, c = B.lib(), cache(B)

    def go(k=P, kt=512, kh=128, v=P, vt=512, vh=128, slots=P, tokens=4):
        return L.kv_append(ctypes.byref(c), k, kt, kh, v, vt, vh, slots, tokens, None)

    for kw in (dict(k=None), dict(slots=None), dict(tokens=0), dict(tokens=1 << 31), dict(kt=64), dict(vh=64),
               dict(kh=-128)):
        assert go(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(k=P + 2), dict(kt=516), dict(vh=132), dict(slots=P + 4)):
        assert go(**kw) == B.FP4_ERR_ALIGNMENT, kw


def test_plan_refusals(B):
    L = B.lib()

    def go(cached=P, new=P + 4096, batch=4, page=64, free=P, nfree=8, table=P, stride=8, maxp=8, total=P + 8192, qs=P,
           slots=P, pos=P, tokens=16, taken=P):
        return L.kv_plan(cached, new, batch, page, free, nfree, table, stride, maxp, total, qs, slots, pos, tokens,
                         taken, None)

    for kw in (dict(page=0), dict(page=24), dict(batch=16385)):
        assert go(**kw) == B.FP4_ERR_UNSUPPORTED, kw
    for kw in (dict(cached=None), dict(table=None), dict(taken=None), dict(batch=0), dict(tokens=0), dict(maxp=0),
               dict(maxp=9), dict(nfree=-1), dict(free=None), dict(total=P), dict(stride=1 << 32)):
        assert go(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(slots=P + 4), dict(new=P + 2), dict(pos=P + 1)):
        assert go(**kw) == B.FP4_ERR_ALIGNMENT, kw


def test_attention_refusals(B):
    L, c = B.lib(), cache(B)
    need = L.kv_attention_workspace_bytes(4, 4, 2, 128, 1)
    assert need > 0

    def go(q=P, qt=512, qh=128, tokens=4, heads=4, qs=P, total=P, batch=4, table=P, stride=8, maxp=8, mq=1, scale=0.1,
           window=0, ws=P, wsb=need, out=P, lse=None):
        return L.kv_attention(ctypes.byref(c), q, qt, qh, tokens, heads, qs, total, batch, table, stride, maxp, mq,
                              scale, window, ws, wsb, out, lse, None)

    for kw in (dict(q=None), dict(qs=None), dict(total=None), dict(table=None), dict(ws=None), dict(out=None),
               dict(tokens=0), dict(batch=0), dict(heads=3), dict(heads=0), dict(maxp=0), dict(stride=7), dict(mq=0),
               dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(wsb=need - 1), dict(qt=100), dict(qh=64)):
        assert go(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(q=P + 8), dict(out=P + 2), dict(ws=P + 4), dict(qt=516), dict(qh=129), dict(lse=P + 2)):
        assert go(**kw) == B.FP4_ERR_ALIGNMENT, kw


def test_workspace_bytes(B):
    f = B.lib().kv_attention_workspace_bytes
    assert f(0, 8, 8, 128, 1) == 0 and f(1, 8, 3, 128, 1) == 0 and f(1, 8, 8, 512, 1) == 0 and f(1, 8, 8, 128, 0) == 0
    assert 0 < f(1, 8, 8, 128, 1) <= f(64, 8, 8, 128, 1)


def test_binding_refuses_tensors_that_do_not_belong_together(B):
    codes = torch.zeros((4, 2, 64, 16), dtype=torch.int32)
    scales = torch.zeros((4, 2, 64, 8), dtype=torch.uint8)
    c = B.kv_cache(codes, scales, codes, scales)
    with pytest.raises(ValueError):
        B.kv_cache(codes, scales, codes, scales, B.MODE_MXFP4)  # scales of the other format
    with pytest.raises(ValueError):
        B.kv_cache(codes, scales, codes[:, :1], scales)
    with pytest.raises(ValueError):
        B.kv_cache(codes.transpose(0, 1), scales, codes, scales)
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.kv_append(c, k, k[:, :1], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.kv_append(c, k, k, torch.zeros(2, dtype=torch.int64))
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.kv_attention(c, k[..., :64], i, i[:3], i.view(1, 4), i)


def refused(name, call, good, **bad):
    """`call` with one argument exchanged is refused, and the message names it."""
    with pytest.raises(ValueError, match=name):
        call(**{**good, **bad})


def test_binding_refuses_tensors_the_kernels_would_misread(B):
    """Types, shapes and layouts are looked at before memory: what is right in all of them but lies on the host is refused last."""
    i32, i64, bf = torch.int32, torch.int64, torch.bfloat16
    ints = lambda *n, dtype=i32: torch.zeros(n, dtype=dtype)  # noqa: E731

    good = dict(cached_lens=ints(4), new_lens=ints(4), free_pages=ints(9), block_table=ints(4, 8), page_size=64, tokens=6)
    with pytest.raises(ValueError, match="GPU"):
        B.kv_plan(**good)
    plan = B.KvPlan(ints(4), ints(5), ints(6, dtype=i64), ints(6), ints())
    with pytest.raises(ValueError, match="GPU"):
        B.kv_plan(**good, plan=plan)
    for name, t in (("cached_lens", ints(4, dtype=i64)), ("new_lens", ints(3)), ("new_lens", ints(4, dtype=i64)),
                    ("new_lens", ints(8)[::2]), ("free_pages", ints(9, dtype=i64)), ("free_pages", ints(9)[::3]), ("block_table", ints(3, 8)),
                    ("block_table", ints(4, 8, dtype=i64)), ("block_table", ints(8, 4).t()), ("block_table", ints(4, 16)[:, ::2])):
        refused(name, B.kv_plan, good, **{name: t})
    for name, t in (("total_lens", ints(3)), ("total_lens", ints(4, dtype=i64)), ("query_start", ints(4)),
                    ("slot_map", ints(6)), ("slot_map", ints(5, dtype=i64)), ("positions", ints(7)), ("pages_taken", ints(2)),
                    ("pages_taken", ints(dtype=i64))):
        refused(name, B.kv_plan, good, plan=plan._replace(**{name: t}))

    codes, scales = torch.zeros((4, 2, 64, 16), dtype=i32), torch.zeros((4, 2, 64, 8), dtype=torch.uint8)
    cache = B.kv_cache(codes, scales, codes, scales)
    refused("global_scale_k", B.kv_cache, dict(k_codes=codes, k_scales=scales, v_codes=codes, v_scales=scales),
            global_scale_k=torch.ones(2))
    refused("global_scale_v", B.kv_cache, dict(k_codes=codes, k_scales=scales, v_codes=codes, v_scales=scales),
            global_scale_v=torch.ones((), dtype=torch.float64))

    good = dict(cache=cache, k=torch.zeros((3, 2, 128), dtype=bf), v=torch.zeros((3, 2, 128), dtype=bf), slot_map=ints(3, dtype=i64))
    with pytest.raises(ValueError, match="GPU"):
        B.kv_append(**good)
    for name, t in (("slot_map", ints(3)), ("slot_map", ints(6, dtype=i64)[::2]), ("k", torch.zeros((3, 2, 128), dtype=torch.float16)),
                    ("v", torch.zeros((3, 2, 128))), ("v", torch.zeros((3, 1, 128), dtype=bf)),
                    ("k", torch.zeros((3, 2, 256), dtype=bf)[..., ::2]), ("k", torch.zeros((3, 256), dtype=bf))):
        refused(name, B.kv_append, good, **{name: t})

    good = dict(cache=cache, q=torch.zeros((3, 4, 128), dtype=bf), query_start=ints(3), total_lens=ints(2), block_table=ints(2, 8),
                ws=torch.zeros(64, dtype=torch.uint8), out=torch.zeros((3, 4, 128), dtype=bf), lse=torch.zeros((3, 4)))
    with pytest.raises(ValueError, match="GPU"):
        B.kv_attention(**good)
    for name, t in (("q", torch.zeros((3, 4, 128), dtype=torch.float16)), ("q", torch.zeros((3, 4, 64), dtype=bf)),
                    ("q", torch.zeros((3, 4, 256), dtype=bf)[..., ::2]), ("query_start", ints(3, dtype=i64)), ("query_start", ints(2)),
                    ("total_lens", ints(2, dtype=i64)), ("total_lens", ints(4)[::2]), ("block_table", ints(1, 8)),
                    ("block_table", ints(8, 2).t()), ("block_table", ints(2, 8, dtype=i64)), ("ws", torch.zeros(64)[::2]),
                    ("out", torch.zeros((3, 4, 128))), ("out", torch.zeros((2, 4, 128), dtype=bf)),
                    ("out", torch.zeros((3, 4, 256), dtype=bf)[..., ::2]), ("lse", torch.zeros((3, 4), dtype=bf)), ("lse", torch.zeros((4, 3)))):
        refused(name, B.kv_attention, good, **{name: t})


def test_workspace_bytes_of_a_head_size_no_call_takes(B):
    f = B.lib().kv_attention_workspace_bytes
    assert f(1, 8, 8, 40, 1) == 0 and f(1, 8, 8, 100, 700) == 0 and f(1, 8, 8, 96, 1) > 0
