"""Plain 64-bit implementations of the operators around a decoder layer's products, and what a kernel in fp32 may make of
them.  Nothing here uses the library; formats are rounded by tables."""
import math

import numpy as np
import torch

GROUP = {2: 16, 1: 32}  # mode -> elements per scale
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array(sorted([m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])[:-1])


def nearest(a, grid):
    """Index of the grid's nearest value to a >= 0, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    below, above = a - grid[hi - 1], grid[hi] - a
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def scale_of(b, mode, gs):
    """Scale bytes of block maxima b >= 0."""
    if mode == 2:
        return nearest(b / (6 * gs), E4M3)
    _, e = np.frexp(np.where(b > 0, b, 1.0))
    return np.where(b > 0, np.clip(e - 3, -127, 127), -127) + 127


def check_codes(codes, scales, y, dy, mode, gs=1.0):
    """codes uint32 [rows, cols/8] and linear scales uint8 [rows, cols/group] are the block rule's for some values within
    dy of y, each block's scale and each element looked at on its own.  The rule's own arithmetic (a quotient, the
    product s8 gs, its reciprocal, a product) is off by at most 2^-24 each: 2^-22 together."""
    g = GROUP[mode]
    rows, cols = y.shape
    lo, hi = np.maximum(np.abs(y) - dy, 0), np.abs(y) + dy
    bl, bh = (v.reshape(rows, -1, g).max(-1) for v in (lo, hi))
    s = scales.astype(np.int64)
    assert np.all((scale_of(bl * (1 - 2.0 ** -22), mode, gs) <= s) & (s <= scale_of(bh * (1 + 2.0 ** -22), mode, gs)))
    step = E4M3[s] * gs if mode == 2 else 2.0 ** (s - 127.0)
    step = np.repeat(step, g, -1)
    nib = np.stack([(codes >> np.uint32(4 * k)) & np.uint32(15) for k in range(8)], -1).reshape(rows, cols).astype(np.int64)
    with np.errstate(divide="ignore", invalid="ignore"):
        vl, vh = (np.where(step > 0, v / step, 0) for v in (lo * (1 - 2.0 ** -22), hi * (1 + 2.0 ** -22)))
    mag = nib & 7
    assert np.all((nearest(vl, E2M1) <= mag) & (mag <= nearest(vh, E2M1)))
    sure = np.abs(y) > dy
    assert np.array_equal((nib >= 8)[sure], (y < 0)[sure])


# ------------------------------------------------------------------- norm


def rms_norm(x, weight=None, eps=1e-6, residual=None):
    """(h, y) in 64 bits."""
    h = x.double().numpy()
    if residual is not None:
        h = h + residual.double().numpy()
    m = (h * h).mean(-1, keepdims=True) + eps
    y = np.where(m > 0, h / np.sqrt(np.where(m > 0, m, 1)), 0.0)
    return h, y if weight is None else y * weight.double().numpy()


# ------------------------------------------------------------------- rope


def frequencies(d, base=10000.0, scaling="none", factor=1.0, original=1, low=1.0, high=32.0):
    f = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "base":
        b = base * factor ** (d / (d - 2.0)) if d > 2 else base
        return [b ** (-2.0 * i / d) for i in range(d // 2)], 1.0
    if scaling == "wavelength":
        out = []
        for x in f:
            wave = 2 * math.pi / x
            if wave < original / high:
                out.append(x)
            elif low > 0 and wave > original / low:
                out.append(x / factor)
            else:
                s = (original / wave - low) / (high - low)
                out.append((1 - s) * x / factor + s * x)
        return out, 1.0
    if scaling == "ramp":
        n = lambda t: d * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        first, last = max(math.floor(n(high)), 0), min(math.ceil(n(low)), d - 1)
        ramp = [min(1.0, max(0.0, (i - first) / max(last - first, 0.001))) for i in range(d // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1
    return f, 1.0


def rope(x, positions, freqs, scale, interleaved, backward=False):
    """(result, bound) in 64 bits: x [tokens, heads, dim] array, bound what an fp32 rotation may be off before its last
    rounding: entries of the table are off by 2^-24 of themselves, so are both products and their sum."""
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(freqs)
    c, s = (np.cos(a) * scale)[:, None], (np.sin(a) * scale * (-1 if backward else 1))[:, None]
    d = 2 * len(freqs)
    i, j = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    out, bound = x.copy(), np.zeros_like(x)
    out[..., i], out[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    # (the reference's own angle is a rounded product: 2^-53 of up to 2^20 radians, and with it cos and sin)
    both = (np.abs(x[..., i]) + np.abs(x[..., j])) * (scale * (3 * 2.0 ** -24 + 2.0 ** -32))
    bound[..., i] = bound[..., j] = both
    return out, bound


# -------------------------------------------------------------------- moe


def moe_sort(ids, experts):
    flat = ids.reshape(-1).astype(np.int64)
    valid = (flat >= 0) & (flat < experts)
    key = np.where(valid, flat, experts)
    order = np.argsort(key, kind="stable")
    slot = np.full(flat.size, -1, np.int64)
    slot[order] = np.arange(flat.size)
    slot[~valid] = -1
    key = key[order]
    return (np.where(key < experts, order // ids.shape[1], 0), np.minimum(key, experts - 1), slot.reshape(ids.shape),
            np.searchsorted(key, np.arange(experts + 1)))


def bf16(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().double().numpy()


def assert_within(got, want, bound, what=""):
    """bf16 results: half a step (2^-8) of rounding on top of `bound`."""
    got = bf16(got)
    off = np.abs(got - want)
    most = 2.0 ** -8 * (np.abs(want) + bound) + bound + 2.0 ** -134
    assert np.all(off <= most), f"{what}: {np.max(off - most)} over at {np.argmax(off - most)}"
