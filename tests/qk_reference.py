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


class _Stored(torch.autograd.Function):
    """A tensor that is kept in bf16, as its gradient is."""

    @staticmethod
    def forward(ctx, x):
        return x.bfloat16().double()

    @staticmethod
    def backward(ctx, g):
        return g.bfloat16().double()


def stack(X, dY, layers, batch, seq, ctx, H, KV, hd, sets, pos, freq, m, dims, layout, eps=1e-5,
          stored=False):
    """One step of a decoder stack with head norms (gains gq, gk where a layer has them) and this
    rotation, by float64 autograd.  sets: per layer the kept (q, k, ffn) channels of the context
    rows, None for all.  stored: every tensor that the step keeps or hands on, and every operand
    of the attention's products, is rounded to bf16, and its gradient too; all else stays float64.
    Returns (y, dX, one dict of LoRA gradients a layer)."""
    bf = _Stored.apply if stored else lambda a: a
    t64 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.float64))  # noqa: E731
    T = batch * seq
    is_ctx = np.concatenate([np.arange(seq) < c for c in ctx])

    def mask(n, idx):
        keep = np.ones((T, n))
        if idx is not None:
            drop = np.setdiff1d(np.arange(n), idx)
            keep[np.ix_(is_ctx, drop)] = 0.0
        return t64(keep)

    def norm(x, g):
        return x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps) * g

    angle = t64(pos)[:, None] * t64(freq)[None]
    c, s = m * torch.cos(angle)[:, None], m * torch.sin(angle)[:, None]
    lo, hi = ((slice(0, dims // 2), slice(dims // 2, dims)) if layout == "half"
              else (slice(0, dims, 2), slice(1, dims, 2)))

    def turn(y, heads, g):
        y = y.view(T, heads, hd)
        if g is not None:
            y = norm(y, g)
        out = y.clone()
        out[..., lo] = y[..., lo] * c - y[..., hi] * s
        out[..., hi] = y[..., lo] * s + y[..., hi] * c
        return bf(out).view(batch, seq, heads, hd).transpose(1, 2)

    x0 = t64(X).requires_grad_()
    x, leaves = x0, []
    causal = torch.ones(seq, seq, dtype=torch.bool).tril()
    for lay, (iq, ik, iff) in zip(layers, sets):
        w = {k: t64(v) for k, v in lay.items() if k != "scale"}
        leaf = {k: w[k].requires_grad_() for k in w if k[0] in "AB"}
        leaves.append(leaf)

        def lin(a, nm):
            return bf(a @ w["W" + nm].T + lay["scale"] * (a @ w["A" + nm].T) @ w["B" + nm].T)

        n1 = bf(norm(x, w["g1"]))
        q = turn(lin(n1, "q") * mask(H * hd, iq), H, w.get("gq"))
        k = turn(lin(n1, "k") * mask(KV * hd, ik), KV, w.get("gk"))
        v = lin(n1, "v").view(batch, seq, KV, hd).transpose(1, 2)
        k, v = (a.repeat_interleave(H // KV, dim=1) for a in (k, v))
        z = q @ k.transpose(-1, -2) / math.sqrt(hd)
        if stored:  # the softmax's derivative is handed on in bf16 too, its statistics are not
            z.register_hook(lambda g: g.bfloat16().double())
        p = bf(z.masked_fill(~causal, -math.inf).softmax(-1))
        h = bf(x + lin(bf(p @ v).transpose(1, 2).reshape(T, H * hd), "o"))
        n2 = bf(norm(h, w["g2"]))
        z = bf(torch.nn.functional.silu(lin(n2, "g")) * lin(n2, "u"))
        x = bf(h + lin(z * mask(z.shape[1], iff), "d"))
    x.backward(t64(dY))
    return (x.detach().numpy(), x0.grad.numpy(),
            [{"d" + k: v.grad.numpy() for k, v in leaf.items()} for leaf in leaves])


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
