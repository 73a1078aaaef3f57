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
