"""GPU: rotation of q and k with optional head norms (slora_qk_rotary_fwd /
_bwd) against float64 formulas, over layouts, scalings, head widths, strides,
positions and sliced rows; gradients against differences; graph replay, other
streams, in-place rows.

Tolerances count roundings: a stored bf16 value is off by half a step, 2^-8
relative; the fp32 work before it (angle 2^-23, products, rsqrt 2^-22, sums of
at most 256 squares) by less than 2^-18 of the terms it adds, which is what an
fp32 result may be off by."""
import ctypes
import decimal
import threading

import numpy as np
import pytest
import torch

from tests import qk_reference as R

pytestmark = pytest.mark.gpu
STORE = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
WORK = 2.0 ** -18


@pytest.fixture(scope="module")
def L():
    from contextual_sparsity_lora_svd_b200 import _lib
    return _lib


def heads_of(t, h):
    a = R.f64(t)
    return a.reshape(a.shape[0], h, -1)


def pair_size(y, dims, layout):
    """Magnitude of each channel's pair: what the rotation's rounding scales with."""
    out = np.abs(y)
    lo, hi = ((slice(0, dims // 2), slice(dims // 2, dims)) if layout == "half"
              else (slice(0, dims, 2), slice(1, dims, 2)))
    p = np.abs(y[..., lo]) + np.abs(y[..., hi])
    out[..., lo] = p
    out[..., hi] = p
    return out


def check(got, want, size, dt, what):
    got = R.f64(got).reshape(want.shape)
    tol = STORE[dt] * np.abs(want) + WORK * size
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - want) / (tol + 1e-300)):.2f} tolerances")


def rand(gen, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)


def run_case(L, dt=torch.bfloat16, gdt=None, b=2, s=5, hq=4, hk=2, hd=64, dims=0, layout="half",
             scaling="none", norm=(True, True), pos=None, seed=0, pad=0, eps=1e-5, **rot):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, gdt = b * s, gdt or dt
    freq, m = R.frequencies(dims or hd, scaling=scaling, **rot)
    rt = L.rotary(layout=layout, dims=dims, scaling=scaling, **rot)
    place = np.tile(np.arange(s), b) if pos is None else pos
    dpos = None if pos is None else torch.tensor(pos, dtype=torch.int32, device="cuda")
    parts, rows_f, rows_b = [], [], []
    for h, nm in ((hq, norm[0]), (hk, norm[1])):
        if not h:
            continue
        n = h * hd
        X = rand(gen, (T, n + pad), dt)[:, :n]
        dY = rand(gen, (T, n + pad), gdt)[:, :n]
        g = rand(gen, (hd,), dt, 0.3) + 1 if nm else None
        Y = torch.full((T, n + pad), 7.0, dtype=dt, device="cuda")
        dX = torch.full((T, n + pad), 7.0, dtype=dt, device="cuda")
        dg = torch.full((hd,), 9.0, device="cuda") if nm else None
        parts.append((h, X, dY, g, Y, dX, dg))
        rows_f.append(L.qk_rows(h, X=X, g=g, Y=Y[:, :n]))
        rows_b.append(L.qk_rows(h, X=X, g=g, dY=dY, dX=dX[:, :n], dg=dg))
    k = (lambda r: r[1] if len(r) > 1 else None)
    L.slora_qk_rotary_fwd(b, s, hd, rows_f[0], k(rows_f), rotary=rt, pos=dpos, eps=eps)
    L.slora_qk_rotary_bwd(b, s, hd, rows_b[0], k(rows_b), rotary=rt, pos=dpos, eps=eps)
    torch.cuda.synchronize()
    d_ = dims or hd
    for i, (h, X, dY, g, Y, dX, dg) in enumerate(parts):
        n = h * hd
        x, gg = heads_of(X, h), None if g is None else R.f64(g)
        want = R.qk_forward(x, gg, eps, place, freq, m, d_, layout)
        check(Y[:, :n], want, pair_size(want, d_, layout), dt, f"Y of tensor {i}")
        dx, sums, size = R.qk_backward(x, gg, eps, heads_of(dY, h), place, freq, m, d_, layout)
        check(dX[:, :n], dx, 4 * pair_size(size, d_, layout), dt,
              f"dX of tensor {i}")
        if pad:  # the columns between the rows stay as they were
            assert (Y[:, n:] == 7).all() and (dX[:, n:] == 7).all()
        if dg is not None:
            # every term has the rounding of its products (WORK of it); the chain of
            # additions of a lane is at most 64 long in these sizes
            err = np.abs(R.f64(dg) - sums[0])
            assert (err <= (WORK + 64 * 2.0 ** -24) * sums[1]).all(), (err / sums[1]).max()
    return parts


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hd,dims", [(64, 0), (128, 64), (128, 32), (80, 20), (96, 24), (256, 0),
                                     (2, 0), (6, 2), (10, 4), (34, 0), (250, 248), (256, 2)])
def test_head_widths_and_parts(L, layout, hd, dims):
    run_case(L, hd=hd, dims=dims, layout=layout)


@pytest.mark.parametrize("dt,gdt", [(torch.bfloat16, torch.float32), (torch.float32, None)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hd,dims", [(128, 0), (96, 24), (18, 6)])
def test_dtypes(L, dt, gdt, layout, hd, dims):
    run_case(L, dt=dt, gdt=gdt, hd=hd, dims=dims, layout=layout)


@pytest.mark.parametrize("scaling,rot", [
    ("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0, base=500000.0)),
    ("bands", dict(factor=8.0, orig_len=8192, base=500000.0)),
    ("bands", dict(factor=4.0, orig_len=512, low=0.5, high=2.0)),
    ("yarn", dict(factor=16.0, orig_len=4096)), ("yarn", dict(factor=2.0, orig_len=64, mscale=1.25)),
    ("yarn", dict(factor=4.0, orig_len=5))])
def test_scalings(L, scaling, rot):
    run_case(L, hd=128, scaling=scaling, dt=torch.float32, **rot)


@pytest.mark.parametrize("b,s,hq,hk", [(1, 1, 1, 1), (1, 1, 32, 8), (1, 1300, 3, 1), (7, 1, 5, 0),
                                       (3, 401, 8, 2), (1, 9, 40, 40), (2, 2500, 1, 0)])
def test_sizes(L, b, s, hq, hk):
    run_case(L, b=b, s=s, hq=hq, hk=hk, hd=64)


@pytest.mark.parametrize("norm", [(True, False), (False, True), (False, False)])
def test_norm_of_either_tensor(L, norm):
    run_case(L, norm=norm, hd=128)


@pytest.mark.parametrize("pad", [8, 4, 2, 1, 64])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strided_rows(L, pad, layout):
    run_case(L, pad=pad, layout=layout, hd=64)


def test_far_negative_and_repeated_positions(L):
    pos = np.array([0, 0, 1, -5, 1_000_000, 2 ** 31 - 1, -2 ** 31, 123_456_789, 3, 3], dtype=np.int64)
    # float64 angles of the reference are off by 2^31 * 2^-53 = 2^-22 rad themselves
    run_case(L, b=2, s=5, pos=pos, hd=128, dt=torch.float32)


def test_zero_head_and_tiny_values(L):
    """A head of zeros has finite output and gradient (eps alone)."""
    hd, T = 64, 3
    X = torch.zeros(T, 2 * hd, dtype=torch.bfloat16, device="cuda")
    X[1, hd:] = 1e-20
    g = torch.ones(hd, dtype=torch.bfloat16, device="cuda")
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    dY = torch.ones_like(X)
    L.slora_qk_rotary_fwd(1, T, hd, L.qk_rows(2, X=X, g=g, Y=Y))
    L.slora_qk_rotary_bwd(1, T, hd, L.qk_rows(2, X=X, g=g, dY=dY, dX=dX))
    assert (Y[0] == 0).all() and torch.isfinite(Y).all() and torch.isfinite(dX).all()
    # at x = 0 the backward is the rotation back times g / sqrt(eps)
    freq, m = R.frequencies(hd)
    want = R.rotate(np.ones((T, 2, hd)), np.arange(T), freq, m, hd, "half", back=True) / 1e-5 ** 0.5
    check(dX, want, pair_size(want, hd, "half"), torch.bfloat16, "dX at zero")


def test_nan_and_infinity_stay_in_their_head(L):
    hd = 64
    X = torch.randn(4, 3 * hd, device="cuda").bfloat16()
    clean = X.clone()
    X[2, hd + 5] = float("nan")
    X[3, 3] = float("inf")
    g = torch.ones(hd, dtype=torch.bfloat16, device="cuda")
    Y, Y0 = torch.empty_like(X), torch.empty_like(X)
    L.slora_qk_rotary_fwd(1, 4, hd, L.qk_rows(3, X=X, g=g, Y=Y))
    L.slora_qk_rotary_fwd(1, 4, hd, L.qk_rows(3, X=clean, g=g, Y=Y0))
    touched = torch.zeros_like(X, dtype=torch.bool)
    touched[2, hd:2 * hd] = True
    touched[3, :hd] = True
    assert torch.equal(Y[~touched], Y0[~touched])
    assert Y[2, hd:2 * hd].isnan().all() and Y[3, 3].isnan()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_and_same_bits(L, layout):
    """Y over X and dX over dY give the bits of separate buffers; a call repeated
    gives its bits again (dg too)."""
    hd, h, T = 128, 5, 700
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    X, dY = rand(gen, (T, h * hd), torch.bfloat16), rand(gen, (T, h * hd), torch.bfloat16)
    g = rand(gen, (hd,), torch.bfloat16)
    rt = L.rotary(layout=layout)
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    dg, dg2 = torch.empty(hd, device="cuda"), torch.empty(hd, device="cuda")
    L.slora_qk_rotary_fwd(1, T, hd, L.qk_rows(h, X=X, g=g, Y=Y), rotary=rt)
    L.slora_qk_rotary_bwd(1, T, hd, L.qk_rows(h, X=X, g=g, dY=dY, dX=dX, dg=dg), rotary=rt)
    X2, dY2 = X.clone(), dY.clone()
    L.slora_qk_rotary_bwd(1, T, hd, L.qk_rows(h, X=X, g=g, dY=dY2, dX=dY2, dg=dg2), rotary=rt)
    L.slora_qk_rotary_fwd(1, T, hd, L.qk_rows(h, X=X2, g=g, Y=X2), rotary=rt)
    assert torch.equal(X2, Y) and torch.equal(dY2, dX) and torch.equal(dg, dg2)
    X3 = X.clone()
    L.slora_qk_rotary_bwd(1, T, hd, L.qk_rows(h, X=X3, g=g, dY=dY, dX=X3), rotary=rt)
    assert torch.equal(X3, dX)


def test_q_and_k_inside_one_fused_buffer(L):
    """q and k as column ranges of one [T x (H + 2 KV) hd] projection output."""
    T, H, KV, hd = 33, 4, 2, 64
    F = torch.randn(T, (H + 2 * KV) * hd, device="cuda").bfloat16()
    keep = F.clone()
    q, k = F[:, :H * hd], F[:, H * hd:(H + KV) * hd]
    L.slora_qk_rotary_fwd(1, T, hd, L.qk_rows(H, X=q, Y=q), L.qk_rows(KV, X=k, Y=k))
    freq, m = R.frequencies(hd)
    for a, o, h in ((q, keep[:, :H * hd], H), (k, keep[:, H * hd:(H + KV) * hd], KV)):
        want = R.rotate(heads_of(o, h), np.arange(T), freq, m, hd, "half")
        check(a, want, pair_size(want, hd, "half"), torch.bfloat16, "fused rows")
    assert torch.equal(F[:, (H + KV) * hd:], keep[:, (H + KV) * hd:])


def test_gradient_against_differences(L):
    """dX and dg of sum(Y * dY) against central differences of the fp32 forward."""
    hd, h, T, eps = 12, 2, 3, 1e-3
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    X, dY = rand(gen, (T, h * hd), torch.float32), rand(gen, (T, h * hd), torch.float32)
    g = rand(gen, (hd,), torch.float32) + 1
    rt = L.rotary(dims=8, layout="interleaved", scaling="yarn", factor=4.0, orig_len=64)
    dX, dg = torch.empty_like(X), torch.empty(hd, device="cuda")
    L.slora_qk_rotary_bwd(1, T, hd, L.qk_rows(h, X=X, g=g, dY=dY, dX=dX, dg=dg), rotary=rt, eps=eps)

    def value(X, g):
        Y = torch.empty_like(X)
        L.slora_qk_rotary_fwd(1, T, hd, L.qk_rows(h, X=X, g=g, Y=Y), rotary=rt, eps=eps)
        return float((Y.double() * dY.double()).sum())

    step = 2.0 ** -7  # truncation step^2 * third derivative (below 10) ~ 6e-4; fp32 noise 1e-6 / step
    for t, i in ((0, 0), (1, 13), (2, 23), (2, 5)):
        up, dn = X.clone(), X.clone()
        up[t, i] += step
        dn[t, i] -= step
        assert abs((value(up, g) - value(dn, g)) / (2 * step) - float(dX[t, i])) < 5e-3
    for i in (0, 7, 11):
        up, dn = g.clone(), g.clone()
        up[i] += step
        dn[i] -= step
        assert abs((value(X, up) - value(X, dn)) / (2 * step) - float(dg[i])) < 5e-3


def sliced(gen, b, s, ctx, heads, hd, idx, dt=torch.bfloat16):
    n, tc = heads * hd, sum(ctx)
    Xc, Xo = rand(gen, (tc, len(idx)), dt), rand(gen, (b * s - tc, n), dt)
    full = torch.zeros(b * s, n, dtype=dt, device="cuda")
    is_ctx = torch.cat([torch.arange(s) < c for c in ctx]).cuda()
    rows = torch.zeros(tc, n, dtype=dt, device="cuda")
    rows[:, idx.long()] = Xc
    full[is_ctx] = rows
    full[~is_ctx] = Xo
    return Xc, Xo, full, is_ctx


@pytest.mark.parametrize("ctx", [[4, 7, 0], [7, 7, 7], [0, 0, 0], [1, 0, 3]])
@pytest.mark.parametrize("layout,hd", [("half", 64), ("interleaved", 64), ("half", 36), ("half", 6)])
@pytest.mark.parametrize("norm", [True, False])
def test_sliced_rows_equal_dense_rows_with_zeros(L, ctx, layout, hd, norm):
    """Sliced rows give the bits of the dense call on rows with zeros in the
    skipped channels (one kernel arithmetic), forward and backward; dg adds the
    same terms in another order (the context rows first): each of the two sums
    of N terms is off by at most N 2^-24 of the terms' magnitudes."""
    b, s, hq, hk = 3, 7, 4, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    rt = L.rotary(layout=layout)
    dense_f, dense_b, sl_f, sl_b, outs = [], [], [], [], []
    for h in (hq, hk):
        n = h * hd
        idx = torch.randperm(n, generator=gen, device="cuda")[:n // 2].int()  # any order
        Xc, Xo, full, is_ctx = sliced(gen, b, s, ctx, h, hd, idx)
        g = rand(gen, (hd,), torch.bfloat16) if norm else None
        dY = rand(gen, (b * s, n), torch.float32)
        Y, Y2, dX = (torch.empty_like(full) for _ in range(3))
        dg, dg2 = (torch.empty(hd, device="cuda") if norm else None for _ in range(2))
        dXc, dXo = torch.full_like(Xc, 5), torch.full_like(Xo, 5)
        dense_f.append(L.qk_rows(h, X=full, g=g, Y=Y))
        dense_b.append(L.qk_rows(h, X=full, g=g, dY=dY, dX=dX, dg=dg))
        sl_f.append(L.qk_rows(h, g=g, Y=Y2, idx=idx, X_ctx=Xc, X_out=Xo))
        sl_b.append(L.qk_rows(h, g=g, dY=dY, idx=idx, X_ctx=Xc, X_out=Xo, dX_ctx=dXc, dX_out=dXo,
                              dg=dg2))
        outs.append((Y, Y2, dX, dXc, dXo, dg, dg2, idx, is_ctx, h, full, g, dY))
    L.slora_qk_rotary_fwd(b, s, hd, *dense_f, rotary=rt)
    L.slora_qk_rotary_bwd(b, s, hd, *dense_b, rotary=rt)
    L.slora_qk_rotary_fwd(b, s, hd, *sl_f, rotary=rt, ctx_len=ctx)
    L.slora_qk_rotary_bwd(b, s, hd, *sl_b, rotary=rt, ctx_len=ctx)
    freq, m = R.frequencies(hd)
    for Y, Y2, dX, dXc, dXo, dg, dg2, idx, is_ctx, h, full, g, dY in outs:
        assert torch.equal(Y, Y2)
        assert torch.equal(dX[is_ctx][:, idx.long()], dXc) and torch.equal(dX[~is_ctx], dXo)
        if norm:
            size = R.qk_backward(heads_of(full, h), R.f64(g), 1e-5, heads_of(dY, h),
                                 np.tile(np.arange(s), b), freq, m, hd, layout)[1][1]
            assert (np.abs(R.f64(dg) - R.f64(dg2)) <= 2 * b * s * h * 2.0 ** -24 * size).all()
    assert L.lib().slora_device_error(1) == 0


@pytest.mark.parametrize("b,s,ctx,parts,hd", [
    (1, 5, [3], [(128, 32768), (128, 20001)], 256),  # the most channels, every one of them kept
    (2, 350, [350, 200], [(8, 500), (2, 250)], 128), (3, 90, [90, 0, 33], [(32, 2048), (8, 512)], 128),
    (65, 11, None, [(4, 100), (1, 31)], 64), (1, 1, [1], [(32, 1), (8, 1024)], 128)])
def test_sliced_rows_of_many_channels(L, b, s, ctx, parts, hd):
    """Whole blocks of rows, lists of two lengths: the dense bits, forward and backward."""
    ctx = ctx or [(5 * i) % (s + 1) for i in range(b)]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(b + s)
    calls, outs = [[], [], [], []], []
    for h, ni in parts:
        n = h * hd
        idx = torch.randperm(n, generator=gen, device="cuda")[:ni].int()
        Xc, Xo, full, is_ctx = sliced(gen, b, s, ctx, h, hd, idx)
        g, dY = rand(gen, (hd,), torch.bfloat16), rand(gen, (b * s, n), torch.float32)
        Y, Y2, dX = (torch.empty_like(full) for _ in range(3))
        dXc, dXo = torch.full_like(Xc, 5), torch.full_like(Xo, 5)
        for c, rows in zip(calls, (
                dict(X=full, Y=Y), dict(X=full, dY=dY, dX=dX), dict(Y=Y2, idx=idx, X_ctx=Xc, X_out=Xo),
                dict(dY=dY, idx=idx, X_ctx=Xc, X_out=Xo, dX_ctx=dXc, dX_out=dXo))):
            c.append(L.qk_rows(h, g=g, **rows))
        outs.append((Y, Y2, dX, dXc, dXo, idx, is_ctx))
    L.slora_qk_rotary_fwd(b, s, hd, *calls[0])
    L.slora_qk_rotary_bwd(b, s, hd, *calls[1])
    L.slora_qk_rotary_fwd(b, s, hd, *calls[2], ctx_len=ctx)
    L.slora_qk_rotary_bwd(b, s, hd, *calls[3], ctx_len=ctx)
    for Y, Y2, dX, dXc, dXo, idx, is_ctx in outs:
        assert torch.equal(Y, Y2)
        assert torch.equal(dX[is_ctx][:, idx.long()], dXc) and torch.equal(dX[~is_ctx], dXo)
    assert L.lib().slora_device_error(1) == 0


def test_sliced_rows_with_no_channels(L):
    """A context row whose head keeps nothing: zero rows, no gradient to write."""
    b, s, h, hd = 1, 6, 2, 64
    Xo = torch.randn(2, h * hd, device="cuda").bfloat16()
    idx = torch.empty(0, dtype=torch.int32, device="cuda")
    Xc = torch.empty(4, 0, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(hd, dtype=torch.bfloat16, device="cuda")
    Y = torch.full((s, h * hd), 3.0, dtype=torch.bfloat16, device="cuda")
    L.slora_qk_rotary_fwd(b, s, hd, L.qk_rows(h, g=g, Y=Y, idx=idx, X_ctx=Xc, X_out=Xo), ctx_len=[4])
    assert (Y[:4] == 0).all() and torch.isfinite(Y).all()


@pytest.mark.parametrize("bad", [[0, 1, 999, 3], [0, 1, -1, 3], [0, 1, 1, 3]])
def test_bad_channel_list_is_reported(L, bad):
    """An entry outside the channels or a repeated one is left out and raised as
    an error flag; nothing outside the buffers is touched."""
    h, hd, T = 1, 64, 5
    idx = torch.tensor(bad, dtype=torch.int32, device="cuda")
    Xc = torch.randn(T, 4, device="cuda").bfloat16()
    Y = torch.empty(T, hd, dtype=torch.bfloat16, device="cuda")
    L.slora_qk_rotary_fwd(1, T, hd, L.qk_rows(h, Y=Y, idx=idx, X_ctx=Xc), ctx_len=[T])
    assert L.lib().slora_device_error(1) == 1
    assert L.lib().slora_device_error(1) == 0
    assert torch.isfinite(Y).all() and (Y[0, 4:32] == 0).all()


def test_many_sequences(L):
    """More sequences than the small launch parameters hold, uneven contexts."""
    b, s, h, hd = 1500, 3, 1, 8
    ctx = [(i * 7) % 4 for i in range(b)]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    idx = torch.tensor([1, 5, 6], dtype=torch.int32, device="cuda")
    Xc, Xo, full, is_ctx = sliced(gen, b, s, ctx, h, hd, idx)
    Y, Y2 = torch.empty_like(full), torch.empty_like(full)
    L.slora_qk_rotary_fwd(b, s, hd, L.qk_rows(h, X=full, Y=Y))
    L.slora_qk_rotary_fwd(b, s, hd, L.qk_rows(h, Y=Y2, idx=idx, X_ctx=Xc, X_out=Xo), ctx_len=ctx)
    assert torch.equal(Y, Y2)


def test_graph_replay_and_other_stream(L):
    """Captured on a side stream and replayed on new inputs: the eager bits."""
    b, s, h, hd = 2, 50, 6, 128
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    X, dY = rand(gen, (b * s, h * hd), torch.bfloat16), rand(gen, (b * s, h * hd), torch.float32)
    g = rand(gen, (hd,), torch.bfloat16)
    Y, dX, dg = torch.empty_like(X), torch.empty_like(X), torch.empty(hd, device="cuda")
    f = L.qk_rows(h, X=X, g=g, Y=Y)
    r = L.qk_rows(h, X=X, g=g, dY=dY, dX=dX, dg=dg)
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def calls():
        L.slora_qk_rotary_fwd(b, s, hd, f, stream=st)
        L.slora_qk_rotary_bwd(b, s, hd, r, ws=ws, stream=st)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        calls()
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            calls()
    X.copy_(rand(gen, X.shape, torch.bfloat16))
    dY.copy_(rand(gen, dY.shape, torch.float32))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (Y, dX, dg)]
    for t in (Y, dX, dg):
        t.zero_()
    torch.cuda.synchronize()
    calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, (Y, dX, dg)))


def test_equals_the_packed_rotation(L):
    """The default form is slora_rope_pack's rotation of dense rows."""
    b, s, h, hd = 2, 40, 3, 128
    X = torch.randn(b * s, h * hd, device="cuda").bfloat16()
    Y, Z = torch.empty_like(X), torch.empty_like(X)
    L.slora_qk_rotary_fwd(b, s, hd, L.qk_rows(h, X=X, Y=Y))
    L.slora_rope_pack(b, s, [s] * b, h * hd, hd, Z, Y=X)
    freq, m = R.frequencies(hd)
    want = R.rotate(heads_of(X, h), np.tile(np.arange(s), b), freq, m, hd, "half")
    for t in (Y, Z):
        check(t, want, pair_size(want, hd, "half"), torch.bfloat16, "rotation")


def same_places(got, want, what):
    """Infinities and NaN where the formula has them, none elsewhere."""
    got = R.f64(got).reshape(want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf]), what
    return np.isfinite(want)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hd,dims", [(64, 32), (96, 48), (80, 20), (128, 8), (24, 4), (36, 34), (48, 20), (10, 4)])
@pytest.mark.parametrize("norm", [False, True])
def test_infinities_in_unrotated_channels_stay_there(L, dt, layout, hd, dims, norm):
    """Channels behind the rotated ones meet no other channel: an infinite or NaN value of one is
    seen by its head's norm alone, and by no other channel's output, gradient or gain gradient."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(hd + dims)
    T, h = 4, 3
    X, dY = rand(gen, (T, h * hd), dt), rand(gen, (T, h * hd), dt)
    g = rand(gen, (hd,), dt, 0.3) + 1 if norm else None
    for t in (X, dY):  # in an even, an odd and the last unrotated channel of different heads
        t[0, dims], t[1, hd + dims + 1], t[2, 3 * hd - 1] = float("inf"), float("nan"), float("-inf")
    rt = L.rotary(layout=layout, dims=dims)
    freq, m = R.frequencies(dims)
    place = np.arange(T)
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    L.slora_qk_rotary_fwd(1, T, hd, L.qk_rows(h, X=X, g=g, Y=Y), rotary=rt)
    gg = None if g is None else R.f64(g)
    with np.errstate(invalid="ignore"):
        want = R.qk_forward(heads_of(X, h), gg, 1e-5, place, freq, m, dims, layout)
    fine = same_places(Y, want, "Y")
    size = np.where(fine, pair_size(np.where(fine, want, 0), dims, layout), 0)
    check(torch.from_numpy(np.where(fine, R.f64(Y).reshape(want.shape), 0)), np.where(fine, want, 0), size, dt, "Y")
    if not norm:
        L.slora_qk_rotary_bwd(1, T, hd, L.qk_rows(h, X=X, dY=dY, dX=dX), rotary=rt)
        want = R.rotate(heads_of(dY, h), place, freq, m, dims, layout, back=True)
        fine = same_places(dX, want, "dX")
        got = torch.from_numpy(np.where(fine, R.f64(dX).reshape(want.shape), 0))
        want = np.where(fine, want, 0)
        check(got, want, pair_size(want, dims, layout), dt, "dX")
        assert torch.equal(dX.view(T, h, hd)[..., dims:].isfinite(), dY.view(T, h, hd)[..., dims:].isfinite())
        return
    dg = torch.empty(hd, device="cuda")  # a clean x under this dY: its heads' dX are lost, the sums are not
    X = rand(gen, (T, h * hd), dt)
    L.slora_qk_rotary_bwd(1, T, hd, L.qk_rows(h, X=X, g=g, dY=dY, dX=dX, dg=dg), rotary=rt)
    bad = torch.zeros(hd, dtype=torch.bool, device="cuda")
    bad[dims], bad[dims + 1], bad[hd - 1] = True, True, True
    assert torch.equal(~dg.isfinite(), bad)


@pytest.mark.parametrize("shapes,kept", [([(32, 128), (8, 128)], 0.5), ([(4, 256), (4, 128)], None)])
def test_calls_from_host_threads(L, shapes, kept):
    """Calls of one kernel whose shared memory differs, from six host threads at once: every one is
    launched and gives its bits (sliced backward of 32 and of 8 heads; dense backward in fp32 of
    heads of 256 and of 128 channels)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    b, s, ctx = 1, 40, [25]
    tok, keep = L.make_tokens(b, s, ctx)
    rot, size, dt = L.rotary(), L.c_sz(0), L.BF16 if kept else L.F32
    jobs = []
    for h, hd in shapes * 3:
        n = h * hd
        if kept:
            idx = torch.randperm(n, generator=gen, device="cuda")[:int(kept * n)].int()
            Xc, Xo, _, _ = sliced(gen, b, s, ctx, h, hd, idx)
            outs = [torch.empty_like(Xc), torch.empty_like(Xo)]
            rows = dict(idx=idx, X_ctx=Xc, X_out=Xo, dX_ctx=outs[0], dX_out=outs[1])
        else:
            outs = [torch.empty(b * s, n, device="cuda")]
            rows = dict(X=rand(gen, (b * s, n), torch.float32), dX=outs[0])
        g = rand(gen, (hd,), torch.bfloat16 if kept else torch.float32)
        rows = L.qk_rows(h, g=g, dY=rand(gen, (b * s, n), torch.float32), **rows)
        stream = torch.cuda.Stream()
        # the C call alone: the binding's Python would hold the interpreter most of the time
        args = (dt, L.F32, ctypes.byref(tok), hd, 1e-5, ctypes.byref(rot), None, ctypes.byref(rows), None, 16,
                ctypes.byref(size), stream.cuda_stream)
        torch.cuda.synchronize()
        assert L.lib().slora_qk_rotary_bwd(*args) == 0
        torch.cuda.synchronize()
        jobs.append((args, rows, stream, outs, [t.clone() for t in outs]))
    failed = []
    start = threading.Barrier(len(jobs))

    def loop(args):
        call = L.lib().slora_qk_rotary_bwd
        start.wait()
        for i in range(5000):
            if call(*args):
                failed.append((i, L._lib_err()))
                return

    threads = [threading.Thread(target=loop, args=(j[0],)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for _, _, _, outs, want in jobs:
        assert all(torch.equal(a, w) for a, w in zip(outs, want))


def exact_cos_sin(pos, base, dims):
    """cos and sin of pos base^(-2p / dims), the angle reduced in 60 digits."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
        ln = decimal.Decimal(base).ln()
        f = [(-ln * 2 * p / dims).exp() for p in range(dims // 2)]
        angle = [[float((decimal.Decimal(int(t)) * v) % (2 * pi)) for v in f] for t in pos]
    a = np.array(angle)
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("base", [10000, 500000])
def test_angles_at_far_positions(L, base):
    """Pairs (1, 0) turned: cosine and sine against angles in 60 digits, to the stated bound.  Of the
    angle in a quarter turn, at most pi / 4, the fixed point's float, its factor and their product are
    rounded by 2^-24 each (1.4e-7 together); the Taylor sums leave 3e-8 and round by less than 2^-23
    (1.2e-7).  The frequency, 2 pi and their quotient are doubles: 3 * 2^-53 of the angle, 4e-16 |pos|."""
    hd = 64
    rng = np.random.default_rng(base)
    pos = np.concatenate([np.arange(40), rng.integers(0, 10 ** 6, 200), rng.integers(-2 ** 31, 2 ** 31, 200),
                          [2 ** 31 - 1, -2 ** 31, 131072, 1 << 20]])
    X = torch.zeros(len(pos), hd, device="cuda")
    X[:, :hd // 2] = 1
    Y = torch.empty_like(X)
    dpos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    L.slora_qk_rotary_fwd(1, len(pos), hd, L.qk_rows(1, X=X, Y=Y), rotary=L.rotary(base=float(base)), pos=dpos)
    c, s = exact_cos_sin(pos, base, hd)
    err = np.maximum(np.abs(R.f64(Y)[:, :hd // 2] - c), np.abs(R.f64(Y)[:, hd // 2:] - s)).max(1)
    assert (err <= 3e-7 + 4e-16 * np.abs(pos)).all(), err.max()
