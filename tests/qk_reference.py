"""Float64 references of the q/k rotation with head norms and of the 8-bit
checkpoints, from their definitions (numpy and torch on the CPU)."""
from __future__ import annotations

import math

import numpy as np
import torch


def frequencies(dims, base=10000.0, scaling="none", factor=1.0, orig_len=0, low=0.0, high=0.0,
                mscale=0.0):
    """(radians per position of each pair, factor on the rotated channels)."""
    i = np.arange(dims // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (dims / (dims - 2))
    f = base ** (-2.0 * i / dims)
    default = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        low, high = (1.0, 4.0) if low == high == 0.0 else (low, high)
        wavelength = 2 * math.pi / f
        keep = np.clip((orig_len / wavelength - low) / (high - low), 0.0, 1.0)
        f = keep * f + (1 - keep) * f / factor
    elif scaling == "yarn":
        low, high = (1.0, 32.0) if low == high == 0.0 else (low, high)
        at = [dims * math.log(orig_len / (2 * math.pi * t)) / (2 * math.log(base))
              for t in (high, low)]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dims - 1)
        ramp = np.clip((i - first) / max(last - first, 0.001), 0.0, 1.0)
        f = ramp * f / factor + (1 - ramp) * f
        default = 0.1 * math.log(factor) + 1.0
    return f, mscale or default


def rotate(y, pos, freq, m, dims, layout, back=False):
    """Rotates heads y [T, heads, hd] (float64 numpy) by pos; back: transposed."""
    angle = pos.astype(np.float64)[:, None] * freq[None]
    c, s = m * np.cos(angle)[:, None], m * np.sin(angle)[:, None]
    if back:
        s = -s
    out = y.copy()
    lo, hi = ((slice(0, dims // 2), slice(dims // 2, dims)) if layout == "half"
              else (slice(0, dims, 2), slice(1, dims, 2)))
    a, b = y[..., lo], y[..., hi]
    out[..., lo] = a * c - b * s
    out[..., hi] = a * s + b * c
    return out


def qk_forward(x, g, eps, pos, freq, m, dims, layout):
    if g is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * g
    return rotate(x, pos, freq, m, dims, layout)


def qk_backward(x, g, eps, dy, pos, freq, m, dims, layout):
    """(dx, dg, bound): bound is the magnitude of the terms that dx is the difference of."""
    dn = rotate(dy, pos, freq, m, dims, layout, back=True)
    if g is None:
        return dn, None, np.abs(dn)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    u = dn * g
    c = r ** 3 * (x * u).mean(-1, keepdims=True)
    terms = dn * x * r
    return r * u - x * c, (terms.sum((0, 1)), np.abs(terms).sum((0, 1))), r * np.abs(u) + np.abs(
        x) * r ** 3 * np.abs(x * u).mean(-1, keepdims=True)


def act8(x):
    """(codes [T x d32], bytes [T x d32/32], values [T x d]) of a checkpoint of x."""
    x = np.asarray(x, dtype=np.float64)
    T, d = x.shape
    d32 = -(-d // 32) * 32
    full = np.zeros((T, d32))
    full[:, :d] = x
    codes = np.zeros((T, d32), dtype=np.int8)
    scales = np.zeros((T, d32 // 32), dtype=np.uint8)
    values = np.zeros((T, d32))
    for t in range(T):
        for b in range(d32 // 32):
            blk = full[t, 32 * b:32 * b + 32]
            if not np.isfinite(blk).all():
                codes[t, 32 * b:32 * b + 32] = 1
                scales[t, b] = 255
                values[t, 32 * b:32 * b + 32] = np.nan
                continue
            top = np.abs(blk).max()
            e = max(math.frexp(top)[1] - 1 if top > 0 else -120, -120)
            q = np.clip(np.rint(blk * 2.0 ** (6 - e)), -127, 127)
            codes[t, 32 * b:32 * b + 32] = q
            scales[t, b] = e + 127
            values[t, 32 * b:32 * b + 32] = q * 2.0 ** (e - 6)
    return codes, scales, values[:, :d]


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()
