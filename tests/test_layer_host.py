"""Host-side checks of the operators around a decoder layer's products (no GPU needed): bad calls are refused before
anything touches a device, and rotary frequencies are what their formulas say."""
import ctypes
import math

import pytest
import torch

import layer_reference as R

P = 256  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def B():
    from block_scaled_fp4_fp_gb300 import build, binding
    build.build()
    binding.lib()
    return binding


def test_rms_norm_refusals(B):
    L = B.lib()

    def go(x=P, xs=64, r=None, rs=0, w=P, eps=1e-6, rows=4, cols=64, so=None, ss=0, out=P + 4096, mode=2, gs=None, xq=None, sc=None,
           layout=0):
        return L.rms_norm(x, xs, r, rs, w, eps, rows, cols, so, ss, out, mode, gs, xq, sc, layout, None)

    for kw in (dict(x=None), dict(out=None), dict(rows=0), dict(rows=1 << 30), dict(cols=0), dict(cols=12), dict(cols=32776, xs=32776),
               dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=2.0), dict(xs=56), dict(r=P, rs=56), dict(so=P + 8192, ss=0),
               dict(xs=1 << 31), dict(r=P, rs=72, so=P, ss=64), dict(so=P, ss=72), dict(out=P, xs=72), dict(out=P + 64, so=P + 64, ss=64),
               dict(r=P + 4096, rs=72), dict(xq=P), dict(xq=P, sc=P, cols=40, xs=40), dict(xq=P, sc=P, mode=1, cols=48, xs=48),
               dict(xq=P, sc=P, mode=1, gs=P), dict(xq=P, sc=P, layout=2)):
        assert go(**kw) == B.FP4_ERR_INVALID_ARG, kw
    assert go(xq=P, sc=P, mode=0) == B.FP4_ERR_UNSUPPORTED
    for kw in (dict(x=P + 8), dict(out=P + 8), dict(w=P + 2), dict(r=P + 4, rs=64), dict(so=P + 8200, ss=64), dict(xs=68),
               dict(r=P, rs=68), dict(xq=P + 2, sc=P), dict(xq=P, sc=P, gs=P + 2)):
        assert go(**kw) == B.FP4_ERR_ALIGNMENT, kw


def rope(B, **kw):
    f = dict(table=P, positions=100, rotary_dim=64, interleaved=0)
    f.update(kw)
    return B.Rope(**f)


BAD_ROPES = [(dict(table=None), "INVALID_ARG"), (dict(positions=0), "INVALID_ARG"), (dict(positions=1 << 31), "INVALID_ARG"),
             (dict(rotary_dim=0), "INVALID_ARG"), (dict(rotary_dim=31), "INVALID_ARG"), (dict(rotary_dim=258), "INVALID_ARG"),
             (dict(rotary_dim=130), "INVALID_ARG"), (dict(table=P + 4), "ALIGNMENT")]


@pytest.mark.parametrize("change,want", BAD_ROPES)
def test_bad_tables_are_refused(B, change, want):
    L, r = B.lib(), rope(B, **change)
    want = getattr(B, "FP4_ERR_" + want)
    cache = B.KvCache(P, P, P, P, None, None, 4, 64, 2, 128, B.MODE_NVFP4)
    assert L.rope(ctypes.byref(r), P, 256, 128, P, 4, 2, 128, 0, P, 256, 128, None) == want
    assert L.kv_append_rope(ctypes.byref(cache), ctypes.byref(r), P, 256, 128, P, 256, 128, P, P, 4, None, 0, 0, 0, None, 0, 0,
                            None) == want


def test_rope_refusals(B):
    L, r = B.lib(), rope(B)

    def go(r=ctypes.byref(r), x=P, xt=256, xh=64, pos=P, tokens=4, heads=2, dim=64, out=P, ot=256, oh=64):
        return L.rope(r, x, xt, xh, pos, tokens, heads, dim, 0, out, ot, oh, None)

    for kw in (dict(r=None), dict(x=None), dict(pos=None), dict(out=None), dict(tokens=0), dict(tokens=1 << 31), dict(heads=0),
               dict(heads=65536), dict(dim=56), dict(dim=68, xh=128, oh=128), dict(dim=264, xh=264, oh=264, xt=600, ot=600), dict(xt=56),
               dict(xh=56), dict(oh=-64), dict(oh=72), dict(ot=128)):
        assert go(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(x=P + 8), dict(out=P + 2), dict(pos=P + 2), dict(out=P + 4096, oh=68), dict(out=P + 4096, ot=260), dict(xt=260, ot=260)):
        assert go(**kw) == B.FP4_ERR_ALIGNMENT, kw


def test_append_rope_refusals(B):
    L, r = B.lib(), rope(B)
    cache = B.KvCache(P, P, P, P, None, None, 4, 64, 2, 128, B.MODE_NVFP4)

    def go(c=ctypes.byref(cache), r=ctypes.byref(r), k=P, kt=512, kh=128, v=P, vt=512, vh=128, slots=P, pos=P, tokens=4, q=None,
           qt=0, qh=0, heads=0, qo=None, qot=0, qoh=0):
        return L.kv_append_rope(c, r, k, kt, kh, v, vt, vh, slots, pos, tokens, q, qt, qh, heads, qo, qot, qoh, None)

    full = dict(q=P, qt=512, qh=128, heads=4, qo=P, qot=512, qoh=128)
    for kw in (dict(c=None), dict(r=None), dict(k=None), dict(slots=None), dict(pos=None), dict(tokens=0), dict(kt=64), dict(vh=64),
               dict(q=P), dict(qo=P), dict(heads=4), dict(full, qo=None), dict(full, heads=0), dict(full, qt=64), dict(full, qoh=136),
               dict(full, qo=P + 4096, qoh=64)):
        assert go(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(k=P + 2), dict(kt=516), dict(slots=P + 4), dict(pos=P + 2), dict(full, q=P + 8), dict(full, qo=P + 4096, qoh=132)):
        assert go(**kw) == B.FP4_ERR_ALIGNMENT, kw
    wide = rope(B, rotary_dim=256)
    assert go(r=ctypes.byref(wide)) == B.FP4_ERR_INVALID_ARG  # more than the cache's head


def test_moe_refusals(B):
    L = B.lib()

    def sort(ids=P, tokens=4, k=2, experts=8, lhs=P + 1024, rhs=P + 2048, slot=P + 3200, off=P + 4096):
        return L.moe_sort(ids, tokens, k, experts, lhs, rhs, slot, off, None)

    for kw in (dict(ids=None), dict(lhs=None), dict(off=None), dict(tokens=0), dict(k=0), dict(k=1025), dict(experts=0), dict(experts=1025),
               dict(tokens=1 << 29, k=3), dict(slot=P)):
        assert sort(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(ids=P + 2), dict(rhs=P + 1), dict(slot=P + 3202)):
        assert sort(**kw) == B.FP4_ERR_ALIGNMENT, kw

    def combine(y=P, rows=8, slot=P, w=P, r=None, tokens=4, k=2, cols=64, out=P + 4096):
        return L.moe_combine(y, rows, slot, w, r, tokens, k, cols, out, None)

    for kw in (dict(y=None), dict(slot=None), dict(out=None), dict(rows=0), dict(tokens=0), dict(k=0), dict(k=1025), dict(cols=12),
               dict(cols=0), dict(out=P)):
        assert combine(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(y=P + 8), dict(out=P + 4), dict(r=P + 2), dict(w=P + 2), dict(slot=P + 1)):
        assert combine(**kw) == B.FP4_ERR_ALIGNMENT, kw

    def back(g=P, y=P, slot=P, w=P, tokens=4, k=2, cols=64, rows=8, used=P, dy=P + 4096, dw=P):
        return L.moe_combine_backward(g, y, slot, w, tokens, k, cols, rows, used, dy, dw, None)

    for kw in (dict(g=None), dict(dy=None), dict(slot=None), dict(y=None), dict(dw=None), dict(cols=20), dict(rows=0), dict(dy=P),
               dict(y=P + 4096)):
        assert back(**kw) == B.FP4_ERR_INVALID_ARG, kw
    for kw in (dict(g=P + 2), dict(dy=P + 8), dict(dw=P + 2), dict(used=P + 2)):
        assert back(**kw) == B.FP4_ERR_ALIGNMENT, kw


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(scaling="wavelength", factor=8.0, original_positions=8192, low=1.0, high=4.0),
            dict(scaling="ramp", factor=16.0, original_positions=4096, low=1.0, high=32.0),
            dict(scaling="ramp", factor=1.0, original_positions=100, low=1.0, high=32.0),
            dict(scaling="ramp", factor=40.0, original_positions=4096, low=0.001, high=2000.0),
            dict(scaling="wavelength", factor=32.0, original_positions=7, low=0.0, high=1000.0)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("dim,base", [(128, 10000.0), (64, 500000.0), (2, 10000.0), (256, 1e6), (34, 100.0)])
def test_frequencies(B, kw, dim, base):
    got, scale = B.rope_frequencies(dim, base, **kw)
    kw = dict(kw)
    if "original_positions" in kw:
        kw["original"] = kw.pop("original_positions")
    want, want_scale = R.frequencies(dim, base, **kw)
    assert len(got) == dim // 2 and got[0] == pytest.approx(want[0], rel=1e-14)
    # a power and a handful of products in fp64: some tens of 2^-53
    assert all(math.isclose(a, b, rel_tol=1e-13, abs_tol=0) for a, b in zip(got, want))
    assert math.isclose(scale, want_scale, rel_tol=1e-15)


def test_frequencies_refusals(B):
    for kw in (dict(rotary_dim=0), dict(rotary_dim=33), dict(rotary_dim=258), dict(base=1.0), dict(base=float("inf")),
               dict(scaling="linear", factor=0.5), dict(scaling="base", factor=float("nan")),
               dict(scaling="ramp", factor=2.0, original_positions=0), dict(scaling="ramp", factor=2.0, low=0.0),
               dict(scaling="wavelength", factor=2.0, low=4.0, high=4.0)):
        with pytest.raises(B.Fp4Error):
            B.rope_frequencies(**{**dict(rotary_dim=64), **kw})
    with pytest.raises(ValueError, match="scaling"):
        B.rope_frequencies(64, scaling="other")
    f = (ctypes.c_double * 32)(*[1.0] * 32)
    L = B.lib()
    assert L.rope_table(f, 64, 1.0, 0, P, None) == B.FP4_ERR_INVALID_ARG
    assert L.rope_table(f, 64, float("nan"), 8, P, None) == B.FP4_ERR_INVALID_ARG
    assert L.rope_table(f, 64, 1.0, 8, P + 4, None) == B.FP4_ERR_ALIGNMENT
    f[3] = float("inf")
    assert L.rope_table(f, 64, 1.0, 8, P, None) == B.FP4_ERR_INVALID_ARG


def refused(name, call, good, **bad):
    """`call` with one argument exchanged is refused, and the message names it."""
    with pytest.raises(ValueError, match=name):
        call(**{**good, **bad})


def test_binding_refuses_tensors_the_kernels_would_misread(B):
    """Types, shapes and layouts are looked at before memory: what is right in all of them but lies on the host is refused last."""
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    z = lambda *n, dtype=bf: torch.zeros(n, dtype=dtype)  # noqa: E731

    good = dict(x=z(4, 64), weight=z(64), residual=z(4, 64), mode=B.MODE_NVFP4, global_scale=z(dtype=f32))
    refused("GPU", B.rms_norm, good)
    for name, t in (("x", z(64)), ("x", z(4, 64, dtype=f32)), ("x", z(4, 128)[:, ::2]), ("weight", z(32)), ("weight", z(64, dtype=f32)),
                    ("residual", z(4, 32)), ("residual", z(64, 4).t()), ("sum_out", z(3, 64)), ("out", z(4, 128)[:, :64]),
                    ("out", z(4, 64, dtype=torch.float16)), ("xq", z(4, 8)), ("xq", z(4, 16, dtype=i32)), ("scales", z(4, 8, dtype=i32)),
                    ("scales", z(4, 2, dtype=torch.uint8)), ("global_scale", z(2, dtype=f32)), ("mode", 0), ("mode", 7)):
        refused(name, B.rms_norm, good, **{name: t})
    refused("mode", B.rms_norm, good, mode=None)

    table = z(10, 32, 2, dtype=f32)
    for t in (z(10, 64, dtype=f32), z(10, 32, 3, dtype=f32), z(10, 32, 2), z(10, 64, 2, dtype=f32)[:, ::2]):
        with pytest.raises(ValueError, match="table"):
            B.rope_from_table(t)
    with pytest.raises(ValueError, match="frequencies"):
        B.rope_table(10, 64, frequencies=[1.0] * 31, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        B.rope_table(10, 64, device="cpu")
    r = B.rope_from_table(table)
    good = dict(rope=r, x=z(3, 4, 64), positions=z(3, dtype=i32))
    refused("GPU", B.rope, good)
    for name, t in (("x", z(3, 256)), ("x", z(3, 4, 64, dtype=f32)), ("x", z(3, 4, 128)[..., ::2]), ("positions", z(4, dtype=i32)),
                    ("positions", z(3, dtype=torch.int64)), ("positions", z(6, dtype=i32)[::2]), ("out", z(3, 4, 32)), ("out", z(3, 4, 64, dtype=f32))):
        refused(name, B.rope, good, **{name: t})

    codes, scales = z(4, 2, 64, 16, dtype=i32), z(4, 2, 64, 8, dtype=torch.uint8)
    good = dict(cache=B.kv_cache(codes, scales, codes, scales), rope=r, k=z(3, 2, 128), v=z(3, 2, 128), slot_map=z(3, dtype=torch.int64),
                positions=z(3, dtype=i32), q=z(3, 4, 128))
    refused("GPU", B.kv_append_rope, good)
    for name, t in (("slot_map", z(3, dtype=i32)), ("positions", z(2, dtype=i32)), ("k", z(3, 2, 64)), ("v", z(3, 2, 128, dtype=f32)),
                    ("v", z(3, 1, 128)), ("q", z(3, 512)), ("q", z(2, 4, 128)), ("q", z(3, 4, 64)), ("q_out", z(3, 3, 128)),
                    ("q_out", z(3, 4, 256)[..., ::2])):
        refused(name, B.kv_append_rope, good, **{name: t})
    refused("q_out", B.kv_append_rope, good, q=None, q_out=z(3, 4, 128))

    good = dict(ids=z(5, 2, dtype=i32), num_experts=4)
    refused("GPU", B.moe_sort, good)
    for t in (z(10, dtype=i32), z(5, 2, dtype=torch.int64), z(2, 5, dtype=i32).t()):
        refused("ids", B.moe_sort, good, ids=t)
    plan = B.MoeSort(z(10, dtype=i32), z(10, dtype=i32), z(5, 2, dtype=i32), z(5, dtype=i32))
    for name, t in (("lhs_idx", z(9, dtype=i32)), ("rhs_idx", z(10)), ("slot", z(10, dtype=i32)), ("offsets", z(4, dtype=i32))):
        refused(name, B.moe_sort, good, plan=plan._replace(**{name: t}))

    good = dict(y=z(10, 64), slot=z(5, 2, dtype=i32), weights=z(5, 2, dtype=f32), residual=z(5, 64))
    refused("GPU", B.moe_combine, good)
    for name, t in (("y", z(640)), ("y", z(10, 64, dtype=f32)), ("y", z(64, 10).t()), ("slot", z(10, dtype=i32)),
                    ("slot", z(5, 2, dtype=torch.int64)), ("weights", z(5, 2)), ("weights", z(2, 5, dtype=f32)), ("residual", z(5, 32)),
                    ("out", z(4, 64)), ("out", z(5, 64, dtype=f32))):
        refused(name, B.moe_combine, good, **{name: t})

    good = dict(dout=z(5, 64), slot=z(5, 2, dtype=i32), weights=z(5, 2, dtype=f32), y=z(10, 64), offsets=z(5, dtype=i32))
    refused("GPU", B.moe_combine_backward, good)
    for name, t in (("dout", z(320)), ("dout", z(4, 64)), ("y", z(10, 32)), ("dy", z(9, 64)), ("dweights", z(5, 2)),
                    ("offsets", z(5, dtype=torch.int64)), ("weights", z(5, 3, dtype=f32))):
        refused(name, B.moe_combine_backward, good, **{name: t})
    refused("dweights", B.moe_combine_backward, good, y=None, dweights=z(5, 2, dtype=f32))


def test_binding_refuses_another_devices_tensors(B, monkeypatch):
    class Elsewhere:
        is_cuda, shape, device = True, (2,), "cuda:1"

        def get_device(self):
            return 1

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        B._need_here(None, Elsewhere())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    B._need_here(None, Elsewhere())


def test_a_single_token_of_heads_before_tokens(B):
    """One token of a long [heads, tokens, head_dim] buffer: a head stride in range is all that its view has, and the library
    takes the strides that the binding gives it (the addresses here are refused behind them)."""
    buffer = torch.empty((64, 300000, 128), dtype=torch.bfloat16, device="meta").transpose(0, 1)
    strides = B._view_strides(buffer[7:8], 1, 64, 128)
    assert strides[1] == 300000 * 128 and B._view_strides(buffer[7:9], 2, 64, 128) == (128, 300000 * 128)
    L, r = B.lib(), rope(B)
    assert L.rope(ctypes.byref(r), P + 2, *strides, P, 1, 64, 128, 0, P + 2, *strides, None) == B.FP4_ERR_ALIGNMENT
    cache = B.KvCache(P, P, P, P, None, None, 4, 64, 64, 128, B.MODE_NVFP4)
    assert L.kv_append_rope(ctypes.byref(cache), ctypes.byref(r), P, *strides, P, *strides, P, P, 1, P + 2, *strides, 64, P + 2, *strides,
                            None) == B.FP4_ERR_ALIGNMENT


def test_no_output_of_a_sort_is_its_ids(B):
    """They are read twice: offsets written over them would change what the second reading finds."""
    L = B.lib()
    good = dict(lhs=P + 1024, rhs=P + 2048, slot=P + 3200, off=P + 4096)
    for name in good:
        b = dict(good, **{name: P})
        assert L.moe_sort(P, 4000, 2, 8, b["lhs"], b["rhs"], b["slot"], b["off"], None) == B.FP4_ERR_INVALID_ARG, name


def test_rotated_queries_do_not_go_over_k_or_v(B):
    """One launch appends K and V and writes the queries: over them, what is appended would depend on which block is first."""
    L, r = B.lib(), rope(B)
    cache = B.KvCache(P, P, P, P, None, None, 4, 64, 2, 128, B.MODE_NVFP4)
    k, v, q = P + 8192, P + 16384, P + 32768

    def go(q_out):
        return L.kv_append_rope(ctypes.byref(cache), ctypes.byref(r), k, 256, 128, v, 256, 128, P, P, 4, q, 256, 128, 2, q_out, 256, 128, None)

    assert go(k) == go(v) == B.FP4_ERR_INVALID_ARG
    assert go(q + 2) == B.FP4_ERR_ALIGNMENT  # (elsewhere the call gets as far as its other checks)
