"""GPU: 8-bit activation checkpoints (slora_act8_pack / _unpack), the RMS norm
that writes and reads them, and the LoRA linear backward from one, against
float64 definitions.  Codes, scale bytes and values are exact; gradients count
the roundings of their stored type and of fp32 sums."""
import numpy as np
import pytest
import torch

from tests import qk_reference as R
from tests.helpers import rel_frob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from contextual_sparsity_lora_svd_b200 import _lib
    return _lib


def rand(gen, shape, dt=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows_in_earnest(gen, T, d, dt):
    """Loud channels, a zero row, wide and subnormal magnitudes."""
    X = torch.randn((T, d), generator=gen, device="cuda")
    X *= torch.exp2(torch.randint(-9, 9, (T, 1), generator=gen, device="cuda").float())
    X[:, ::17] *= 50
    if T > 2:
        X[1] = 0
        X[2] *= 2.0 ** -125
    return X.to(dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 32), (3, 31), (5, 33), (7, 688), (2, 4096), (13, 100),
                                 (1, 4097), (260, 8)])
def test_pack_and_unpack_are_exact(L, dt, T, d):
    X = rows_in_earnest(gen_of(T + d), T, d, dt)
    codes, scales = L.act8_empty(T, d)
    codes.fill_(77)
    scales.fill_(77)
    L.slora_act8_pack(X, codes, scales)
    c, b, v = R.act8(R.f64(X))
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), b)
    for out in (torch.bfloat16, torch.float32):
        Y = torch.full((T, d), 9.0, dtype=out, device="cuda")
        L.slora_act8_unpack(codes, scales, Y)
        assert np.array_equal(R.f64(Y), v)
    # the error bound of the format: 2^-7 of the block's largest magnitude
    pad = np.zeros((T, codes.shape[1]))
    pad[:, :d] = R.f64(X)
    err = np.zeros_like(pad)
    err[:, :d] = np.abs(v - R.f64(X))
    top = np.abs(pad).reshape(T, -1, 32).max(2)
    assert (err.reshape(T, -1, 32).max(2) <= np.maximum(top * 2.0 ** -7, 2.0 ** -127)).all()


def test_ties_and_saturation(L):
    X = torch.zeros(2, 32, device="cuda")
    X[0, :6] = torch.tensor([64.0, 0.5, 1.5, 2.5, -0.5, -1.5])  # step 1: ties to even
    X[1, :4] = torch.tensor([127.75, -127.75, 127.4, 126.5])     # past 127: saturated
    codes, scales = L.act8_empty(2, 32)
    L.slora_act8_pack(X, codes, scales)
    assert codes[0, :6].tolist() == [64, 0, 2, 2, 0, -2] and scales[0, 0] == 133
    assert codes[1, :4].tolist() == [127, -127, 127, 126]


def test_infinities_and_nan_mark_their_block(L):
    X = torch.randn(3, 96, device="cuda").bfloat16()
    X[0, 40] = float("inf")
    X[1, 3] = float("nan")
    X[2, 95] = float("-inf")
    codes, scales = L.act8_empty(3, 96)
    L.slora_act8_pack(X, codes, scales)
    Y = torch.empty_like(X)
    L.slora_act8_unpack(codes, scales, Y)
    nan = torch.zeros(3, 3, dtype=torch.bool, device="cuda")
    nan[0, 1] = nan[1, 0] = nan[2, 2] = True
    assert torch.equal(Y.view(3, 3, 32).isnan().all(2), nan)
    assert torch.equal(Y.view(3, 3, 32).isnan().any(2), nan)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [1, 8, 24])
def test_strided_rows(L, dt, pad):
    T, d = 9, 72
    B = rows_in_earnest(gen_of(1), T, d + pad, dt)
    codes, scales = L.act8_empty(T, d)
    L.slora_act8_pack(B[:, :d], codes, scales)
    c, b, v = R.act8(R.f64(B[:, :d]))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), b)
    out = torch.full((T, d + pad), 4.0, dtype=dt, device="cuda")
    L.slora_act8_unpack(codes, scales, out[:, :d])
    assert np.array_equal(R.f64(out[:, :d]), v) and (out[:, d:] == 4).all()


def test_large_checkpoint_on_another_stream(L):
    """More chunks than one wave, packed on a side stream while another runs."""
    T, d = 3001, 5000
    X = rand(gen_of(3), (T, d))
    codes, scales = L.act8_empty(T, d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    L.slora_act8_pack(X, codes, scales, stream=st)
    st.synchronize()
    rows = [0, 1, 1500, 3000]
    c, b, _ = R.act8(R.f64(X[rows]))
    assert np.array_equal(codes[rows].cpu().numpy(), c)
    assert np.array_equal(scales[rows].cpu().numpy(), b)


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,d", [(1, 8), (5, 688), (3, 1032), (2, 4096), (70, 2040), (2, 8200),
                                 (2, 16384)])
@pytest.mark.parametrize("res", [True, False])
def test_norm_writes_its_checkpoints(L, T, d, res):
    gen = gen_of(d)
    X, A, g = rand(gen, (T, d)), rand(gen, (T, d)) if res else None, rand(gen, (d,))
    H, N, rstd = torch.empty_like(X), torch.empty_like(X), torch.empty(T, device="cuda")
    H2, N2, rstd2 = torch.empty_like(X), torch.empty_like(X), torch.empty(T, device="cuda")
    H8, N8 = L.act8_empty(T, d), L.act8_empty(T, d)
    L.slora_rmsnorm_fwd(X, g, N=N, A=A, H=H if res else None, rstd=rstd)
    L.slora_rmsnorm_fwd_act8(X, g, N2, rstd2, A=A, H=H2 if res else None, H8=H8, N8=N8)
    assert torch.equal(N, N2) and torch.equal(rstd, rstd2)
    if res:
        assert torch.equal(H, H2)
    for ck, src in ((H8, H if res else X), (N8, N)):
        want = L.act8_empty(T, d)
        L.slora_act8_pack(src, *want)
        assert torch.equal(ck[0], want[0]) and torch.equal(ck[1], want[1])
    # one of the two alone
    H9, N9 = L.act8_empty(T, d), L.act8_empty(T, d)
    L.slora_rmsnorm_fwd_act8(X, g, N2, A=A, H=H2 if res else None, H8=H9)
    L.slora_rmsnorm_fwd_act8(X, g, N2, A=A, N8=N9)
    assert torch.equal(H8[0], H9[0]) and torch.equal(N8[0], N9[0])


@pytest.mark.parametrize("T,d", [(3, 2600), (700, 5120), (2, 6144), (400, 8192), (3, 9216), (300, 11008),
                                 (2, 12296), (300, 14336)])
def test_rows_of_several_parts_have_the_plain_bits(L, T, d):
    gen = gen_of(d)
    X, A, g = rand(gen, (T, d)), rand(gen, (T, d)), rand(gen, (d,))
    dN, dRes = [rand(gen, (T, d)) for _ in range(3)], rand(gen, (T, d))
    H, N, H2, N2, dX, dX2 = (torch.empty_like(X) for _ in range(6))
    r, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    H8, N8, want = L.act8_empty(T, d), L.act8_empty(T, d), L.act8_empty(T, d)
    L.slora_rmsnorm_fwd(X, g, N=N, A=A, H=H, rstd=r)
    L.slora_rmsnorm_fwd_act8(X, g, N2, r2, A=A, H=H2, H8=H8, N8=N8)
    assert torch.equal(H, H2) and torch.equal(N, N2) and torch.equal(r, r2)
    for got, src in ((H8, H), (N8, N)):
        L.slora_act8_pack(src, *want)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    V = torch.empty_like(X)
    L.slora_act8_unpack(*H8, V)
    L.slora_rmsnorm_bwd(V, r, g, dN[0], dX, dN1=dN[1], dN2=dN[2], dRes=dRes)
    L.slora_rmsnorm_bwd_act8(H8, r, g, dN[0], dX2, dN1=dN[1], dN2=dN[2], dRes=dRes)
    assert torch.equal(dX, dX2)


@pytest.mark.parametrize("T,d", [(1, 8), (5, 688), (3, 1032), (9, 4096), (2, 8200), (2, 16384)])
@pytest.mark.parametrize("extra", [0, 1, 2])
def test_norm_backward_reads_its_checkpoint(L, T, d, extra):
    """The bits of slora_rmsnorm_bwd on the checkpoint's values, and float64."""
    gen = gen_of(d + extra)
    X, g = rand(gen, (T, d)), rand(gen, (d,))
    dN = [rand(gen, (T, d)) for _ in range(1 + extra)] + [None] * (2 - extra)
    dRes = rand(gen, (T, d)) if extra else None
    H8 = L.act8_empty(T, d)
    L.slora_act8_pack(X, *H8)
    V = torch.empty_like(X)
    L.slora_act8_unpack(*H8, V)
    x = R.f64(X)
    rstd = torch.tensor(1 / np.sqrt((x ** 2).mean(1) + 1e-5), dtype=torch.float32, device="cuda")
    dX, dX2 = torch.empty_like(X), torch.empty_like(X)
    L.slora_rmsnorm_bwd_act8(H8, rstd, g, dN[0], dX, dN1=dN[1], dN2=dN[2], dRes=dRes)
    L.slora_rmsnorm_bwd(V, rstd, g, dN[0], dX2, dN1=dN[1], dN2=dN[2], dRes=dRes)
    assert torch.equal(dX, dX2)
    v, r = R.f64(V), R.f64(rstd)[:, None]
    u = sum(R.f64(t) for t in dN if t is not None) * R.f64(g)
    c = r ** 3 * (u * v).mean(1, keepdims=True)
    base = 0 if dRes is None else R.f64(dRes)
    want = base + r * u - v * c
    # half a bf16 step of the result; the fp32 sum of d terms within 2^-16 of their magnitudes
    size = np.abs(base) + r * np.abs(u) + np.abs(v) * r ** 3 * np.abs(u * v).mean(1, keepdims=True)
    assert (np.abs(R.f64(dX) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * size).all()


# -------------------------------------------------------- linear backward
def linear_case(L, side, b, s, ctx, k, n, r, ni, seed=0, scale=2.0, idx=None):
    """One call against float64; returns the outputs."""
    gen = gen_of(seed)
    T, TC = b * s, sum(ctx)
    is_ctx = np.concatenate([np.arange(s) < c for c in ctx])
    W = rand(gen, (n, k), scale=k ** -0.5)
    A, B = rand(gen, (r, k), scale=k ** -0.5), rand(gen, (n, r), scale=0.1)
    cols = {"none": n, "out_rows": n, "in_cols": k}[side]
    if side != "none" and idx is None:
        pick = torch.randperm(cols, generator=gen, device="cuda")[:ni]
        idx = torch.sort(pick).values.int()
    empty = lambda t: t if t.numel() else None
    x = np.zeros((T, k))
    dy = np.zeros((T, n))
    if side == "in_cols":
        Xc, Xo = rand(gen, (TC, ni)), rand(gen, (T - TC, k))
        X8, O8 = L.act8_empty(TC, ni), L.act8_empty(T - TC, k)
        if Xc.numel():
            L.slora_act8_pack(Xc, *X8)
            rows = np.zeros((TC, k))
            rows[:, R.f64(idx).astype(int)] = R.act8(R.f64(Xc))[2]
            x[is_ctx] = rows
        if Xo.numel():
            L.slora_act8_pack(Xo, *O8)
            x[~is_ctx] = R.act8(R.f64(Xo))[2]
        dYc, dYo = rand(gen, (T, n)), None
        dy = R.f64(dYc)
        dXc, dXo = torch.full_like(Xc, 3), torch.full_like(Xo, 3)
    else:
        X = rand(gen, (T, k))
        X8, O8 = L.act8_empty(T, k), None
        L.slora_act8_pack(X, *X8)
        x = R.act8(R.f64(X))[2]
        nc, rc = (n, T) if side == "none" else (ni, TC)
        dYc, dYo = rand(gen, (rc, nc)), rand(gen, (T - rc, n))
        if side == "none":
            dy = R.f64(dYc)
        else:
            rows = np.zeros((TC, n))
            rows[:, R.f64(idx).astype(int)] = R.f64(dYc)
            dy[is_ctx], dy[~is_ctx] = rows, R.f64(dYo)
        dXc, dXo = torch.full_like(X, 3), None
    XA = rand(gen, (T, r), torch.float32)
    dA, dB = torch.full((r, k), 3.0, device="cuda"), torch.full((n, r), 3.0, device="cuda")
    Wd = W.t().contiguous() if side == "in_cols" else W
    code = {"none": L.SLICE_NONE, "out_rows": L.SLICE_OUT_ROWS, "in_cols": L.SLICE_IN_COLS}[side]
    L.slora_linear_bwd_act8(code, b, s, ctx, k, n, Wd, A, B, scale, idx, X8, XA, dYc, dXc, dA, dB,
                            X8_out=O8, dY_out=None if dYo is None else empty(dYo), dX_out=dXo)
    torch.cuda.synchronize()
    w, a, bb, xa = R.f64(W), R.f64(A), R.f64(B), R.f64(XA)
    p = dy @ bb
    want = dy @ w + scale * p @ a
    got = np.zeros((T, k))
    if side == "in_cols":
        sel = R.f64(idx).astype(int)
        got, mask = np.zeros((T, k)), np.zeros((T, k), dtype=bool)
        if TC and ni:
            block = np.zeros((TC, k))
            block[:, sel] = R.f64(dXc)
            got[is_ctx] = block
            m = np.zeros((TC, k), dtype=bool)
            m[:, sel] = True
            mask[is_ctx] = m
        if T - TC:
            got[~is_ctx] = R.f64(dXo)
            mask[~is_ctx] = True
        want = want * mask
    else:
        got = R.f64(dXc)
    # dX in bf16: half a step of the result and the LoRA part's operand in bf16
    # (2^-8 each of its terms), in the 2-norm well inside 2^-7
    assert rel_frob(got, want) <= 2.0 ** -7
    # fp32 gradients: dYB and the sums in fp32 (tensor-core sums of K or M terms,
    # three bf16 terms of an fp32 operand to 2^-24): 1e-5 in the 2-norm
    assert rel_frob(R.f64(dA), scale * p.T @ x) <= 1e-5
    assert rel_frob(R.f64(dB), scale * dy.T @ xa) <= 1e-5
    return dXc, dA, dB


@pytest.mark.parametrize("side", ["none", "out_rows", "in_cols"])
@pytest.mark.parametrize("b,s,ctx,k,n,r", [
    (1, 1, [1], 64, 64, 8), (2, 9, [4, 7], 72, 152, 5), (1, 300, [200], 688, 256, 16),
    (3, 90, [90, 0, 33], 256, 688, 32), (1, 130, [100], 136, 72, 64), (2, 700, [500, 400], 520, 264, 1),
    (1, 16, [16], 128, 64, 17)])
def test_linear_backward(L, side, b, s, ctx, k, n, r):
    cols = {"none": 0, "out_rows": n, "in_cols": k}[side]
    linear_case(L, side, b, s, ctx, k, n, r, cols // 2)


@pytest.mark.parametrize("side", ["out_rows", "in_cols"])
@pytest.mark.parametrize("ctx,ni", [([0, 0], 20), ([40, 40], 33), ([17, 40], 0), ([40, 40], 0),
                                    ([1, 0], 1), ([23, 31], 72)])
def test_linear_backward_empty_parts(L, side, ctx, ni):
    linear_case(L, side, 2, 40, ctx, 72, 72, 8, ni)


@pytest.mark.parametrize("side", ["none", "out_rows", "in_cols"])
@pytest.mark.parametrize("b,s", [(64, 5), (65, 5), (1500, 3)])
def test_linear_backward_many_sequences(L, side, b, s):
    """Around the number of sequences that the small launch parameters hold, uneven contexts."""
    linear_case(L, side, b, s, [(7 * i) % (s + 1) for i in range(b)], 72, 136, 8, 40)


@pytest.mark.parametrize("side", ["out_rows", "in_cols"])
@pytest.mark.parametrize("last", [104, 2 ** 31 - 1])
def test_linear_backward_leaves_channels_outside_out(L, side, last):
    """An entry outside the weight counts as a channel of zeros and raises the error flag."""
    b, s, ctx, k, n, r = 2, 20, [15, 9], 104, 104, 8
    gen = gen_of(4)
    T, TC = b * s, sum(ctx)
    W, A, B = rand(gen, (104, 104)), rand(gen, (r, k)), rand(gen, (n, r))
    XA = rand(gen, (T, r), torch.float32)
    code = L.SLICE_OUT_ROWS if side == "out_rows" else L.SLICE_IN_COLS
    xs = rand(gen, (T, k)), rand(gen, (TC, 4)), rand(gen, (T - TC, k))
    dys = rand(gen, (TC, 4)), rand(gen, (T - TC, n)), rand(gen, (T, n))
    outs = []
    for keep in (4, 3):
        idx = torch.tensor([2, 5, 60, last][:keep], dtype=torch.int32, device="cuda")
        dA, dB = torch.full((r, k), 7.0, device="cuda"), torch.full((n, r), 7.0, device="cuda")
        ck = []
        for x in (xs[0], xs[1], xs[2]):
            ck.append(L.act8_empty(*x.shape))
            L.slora_act8_pack(x, *ck[-1])
        if keep == 3:  # the values that the four channels' checkpoint holds, of three of them
            v = torch.empty_like(xs[1])
            L.slora_act8_unpack(*ck[1], v)
            ck[1] = L.act8_empty(TC, 3)
            L.slora_act8_pack(v[:, :3].contiguous(), *ck[1])
        if side == "out_rows":
            dX = torch.empty_like(xs[0])
            L.slora_linear_bwd_act8(code, b, s, ctx, k, n, W, A, B, 0.5, idx, ck[0], XA,
                                    dys[0][:, :keep].contiguous(), dX, dA, dB, dY_out=dys[1])
            outs.append((dX, dA, dB))
        else:
            dXc, dXo = torch.full((TC, keep), 7.0, device="cuda").bfloat16(), torch.empty_like(xs[2])
            L.slora_linear_bwd_act8(code, b, s, ctx, k, n, W, A, B, 0.5, idx, ck[1], XA, dys[2], dXc, dA,
                                    dB, X8_out=ck[2], dX_out=dXo)
            if keep == 4:
                assert (dXc[:, 3] == 0).all()
            outs.append((dXc[:, :3], dXo, dA, dB))
        assert L.lib().slora_device_error(1) == (1 if keep == 4 else 0)
        assert L.lib().slora_device_error(1) == 0
    for got, want in zip(*outs):  # the same terms and zeros, in fp32 sums of fewer than 128 terms
        tol = 2.0 ** -8 if got.dtype == torch.bfloat16 else 128 * 2.0 ** -24
        err = rel_frob(R.f64(got), R.f64(want))
        assert err <= tol


def test_linear_backward_is_the_bf16_call_on_the_values(L):
    """dX has the bits of slora_linear_bwd (which does not read the activation
    for it); the gradients agree to that call's bf16 operands."""
    b, s, ctx, k, n, r = 2, 200, [150, 120], 256, 384, 16
    gen = gen_of(9)
    T = b * s
    W, A, B = rand(gen, (n, k)), rand(gen, (r, k)), rand(gen, (n, r))
    X, dY, XA = rand(gen, (T, k)), rand(gen, (T, n)), rand(gen, (T, r), torch.float32)
    X8 = L.act8_empty(T, k)
    L.slora_act8_pack(X, *X8)
    V = torch.empty_like(X)
    L.slora_act8_unpack(*X8, V)
    o = [[torch.empty_like(X), torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")]
         for _ in range(3)]
    for i in range(2):
        L.slora_linear_bwd_act8(L.SLICE_NONE, b, s, ctx, k, n, W, A, B, 0.5, None, X8, XA, dY, *o[i])
    L.slora_linear_bwd(L.SLICE_NONE, b, s, ctx, k, n, W, A, B, 0.5, None, V, XA, dY, *o[2])
    assert all(torch.equal(x, y) for x, y in zip(o[0], o[1]))  # the same bits again
    assert torch.equal(o[0][0], o[2][0])
    for i in (1, 2):
        assert rel_frob(R.f64(o[0][i]), R.f64(o[2][i])) <= 2.0 ** -8


def test_linear_backward_large_split(L):
    """Many tokens and few channels: partial sums of many blocks, same bits twice."""
    x = [linear_case(L, "none", 1, 6000, [4000], 64, 64, 16, 0, seed=3) for _ in range(2)]
    assert all(torch.equal(p, q) for p, q in zip(*x))


def test_linear_backward_captured(L):
    """Captured and replayed twice: the eager bits (counters are left ready)."""
    b, s, ctx, k, n, r = 1, 1024, [700], 512, 256, 16
    gen = gen_of(5)
    T = b * s
    W, A, B = rand(gen, (n, k)), rand(gen, (r, k)), rand(gen, (n, r))
    X, dY, XA = rand(gen, (T, k)), rand(gen, (T, n)), rand(gen, (T, r), torch.float32)
    X8 = L.act8_empty(T, k)
    out = [torch.empty_like(X), torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step(st=None):
        L.slora_act8_pack(X, *X8, stream=st)
        L.slora_linear_bwd_act8(L.SLICE_NONE, b, s, ctx, k, n, W, A, B, 0.5, None, X8, XA, dY, *out,
                                ws=ws, stream=st)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            step(st)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want))
    assert L.lib().slora_device_error(1) == 0


def test_calls_follow_one_another_without_waiting(L):
    """A kernel may be placed while the one before it ends: chains on one stream, in which every
    call reads what the last one wrote and overwrites what it read, and the same chains on four
    streams at once, give the serial bits."""
    def chain(seed, T, k, n, r=16):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        bf = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
        W, A, B, X = bf(n, k), bf(r, k), bf(n, r), bf(T, k)
        XA = torch.randn(T, r, device="cuda", generator=gen)
        c, Y, dX = L.act8_empty(T, k), bf(T, k), bf(T, k)
        dA, dB = torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")
        dY = bf(T, n)
        need = 1 << 25
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def run(stream):
            Y.copy_(X)
            for _ in range(3):
                L.slora_act8_pack(Y, *c, stream=stream)
                L.slora_linear_bwd_act8(L.SLICE_NONE, 1, T, [T], k, n, W, A, B, 0.5, None, c, XA, dY, dX,
                                        dA, dB, ws=ws, stream=stream)
                L.slora_act8_pack(dX, *c, stream=stream)
                L.slora_act8_unpack(*c, Y, stream=stream)
            return Y, dX, dA, dB
        return run

    chains = [chain(1, 512, 1024, 768), chain(2, 77, 688, 256), chain(3, 300, 256, 688), chain(4, 512, 512, 512)]
    want = []
    for f in chains:
        outs = f(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(20):
        got = []
        for f, st in zip(chains, streams):
            with torch.cuda.stream(st):
                got.append(f(st))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert L.lib().slora_device_error(1) == 0


def test_scratch_of_a_call_on_another_stream_is_kept(L):
    """Workspace that the binding takes for a call on a side stream is not handed out again before
    that call has run: the current stream allocates and overwrites as much meanwhile."""
    T, k, n, r = 256, 512, 384, 16
    gen = gen_of(12)
    W, A, B = rand(gen, (n, k)), rand(gen, (r, k)), rand(gen, (n, r))
    X, dY, XA = rand(gen, (T, k)), rand(gen, (T, n)), rand(gen, (T, r), torch.float32)
    X8 = L.act8_empty(T, k)
    L.slora_act8_pack(X, *X8)
    outs = []
    for _ in range(6):
        outs.append((torch.empty_like(X), torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        stream = None
        if i:
            stream = side
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)  # about a millisecond in which the call has not begun
        L.slora_linear_bwd_act8(L.SLICE_NONE, 1, T, [T], k, n, W, A, B, 0.5, None, X8, XA, dY, *o, stream=stream)
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
                for size in (1 << 14, 1 << 16, 1 << 18, 1 << 20, 1 << 21) for _ in range(4)]
        del junk
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    assert L.lib().slora_device_error(1) == 0


@pytest.mark.parametrize("side", ["none", "out_rows", "in_cols"])
def test_linear_gradients_against_differences(L, side):
    """dX, dA and dB of sum(Y dY), Y the sliced forward in float64 on the checkpoint's values: Y is
    linear in each of them, so a central difference is exact; the tolerances are linear_case's."""
    b, s, ctx, k, n, r, scale = 2, 6, [4, 3], 64, 72, 8, 0.75
    gen = gen_of(21)
    T, TC = b * s, sum(ctx)
    is_ctx = np.concatenate([np.arange(s) < c for c in ctx])
    cols = k if side == "in_cols" else n
    idx = torch.sort(torch.randperm(cols, generator=gen, device="cuda")[:24]).values.int()
    sel = R.f64(idx).astype(int)
    W, A, B = rand(gen, (n, k), scale=0.125), rand(gen, (r, k), scale=0.125), rand(gen, (n, r), scale=0.1)
    X, dY = rand(gen, (T, k)), rand(gen, (T, n))
    keep = torch.from_numpy(is_ctx).cuda()
    if side == "in_cols":
        parts = [X[keep][:, idx.long()].contiguous(), X[~keep].contiguous()]
    else:
        parts = [X]
    cks = []
    x = np.zeros((T, k))
    for t in parts:
        cks.append(L.act8_empty(*t.shape))
        L.slora_act8_pack(t, *cks[-1])
    if side == "in_cols":
        rows = np.zeros((TC, k))
        rows[:, sel] = R.act8(R.f64(parts[0]))[2]
        x[is_ctx], x[~is_ctx] = rows, R.act8(R.f64(parts[1]))[2]
    else:
        x = R.act8(R.f64(X))[2]
    w, dy = R.f64(W), R.f64(dY)
    drop = np.setdiff1d(np.arange(cols), sel)

    def value(x, a, bb):
        x = x.copy()
        if side == "in_cols":
            x[np.ix_(is_ctx, drop)] = 0
        y = x @ w.T + scale * (x @ a.T) @ bb.T
        if side == "out_rows":
            y[np.ix_(is_ctx, drop)] = 0
        return (y * dy).sum()

    a64, b64 = R.f64(A), R.f64(B)
    XA = torch.from_numpy(x @ a64.T).float().cuda()
    dA, dB = torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")
    code = {"none": L.SLICE_NONE, "out_rows": L.SLICE_OUT_ROWS, "in_cols": L.SLICE_IN_COLS}[side]
    dXs = [torch.empty_like(t) for t in parts]
    kw, dYc, Wd = {}, dY, W
    if side == "out_rows":
        dYc = dY[keep][:, idx.long()].contiguous()
        kw = dict(dY_out=dY[~keep].contiguous())
    elif side == "in_cols":
        Wd = W.t().contiguous()
        kw = dict(X8_out=cks[1], dX_out=dXs[1])
    L.slora_linear_bwd_act8(code, b, s, ctx, k, n, Wd, A, B, scale, None if side == "none" else idx, cks[0], XA,
                            dYc, dXs[0], dA, dB, **kw)
    got = np.zeros((T, k))
    if side == "in_cols":
        block = np.zeros((TC, k))
        block[:, sel] = R.f64(dXs[0])
        got[is_ctx], got[~is_ctx] = block, R.f64(dXs[1])
    else:
        got = R.f64(dXs[0])

    def differences(which, m):
        out = np.zeros(m.shape)
        for i in np.ndindex(m.shape):
            args = [x, a64, b64]
            args[which] = m.copy()
            args[which][i] += 1.0
            up = value(*args)
            args[which][i] -= 2.0
            out[i] = (up - value(*args)) / 2
        return out

    assert rel_frob(got, differences(0, x)) <= 2.0 ** -7
    assert rel_frob(R.f64(dA), differences(1, a64)) <= 1e-5
    assert rel_frob(R.f64(dB), differences(2, b64)) <= 1e-5


def test_norm_gradient_against_differences(L):
    """dX of sum(N dN) at the checkpoint's values, against central differences of the float64 norm:
    truncation 1e-8, half a bf16 step of the result and the fp32 sum of d terms."""
    T, d = 3, 72
    gen = gen_of(31)
    X, g, dN = rand(gen, (T, d)), rand(gen, (d,)), rand(gen, (T, d))
    H8, N, N8 = L.act8_empty(T, d), torch.empty_like(X), L.act8_empty(T, d)
    rstd, dX = torch.empty(T, device="cuda"), torch.empty_like(X)
    L.slora_act8_pack(X, *H8)
    V = torch.empty_like(X)
    L.slora_act8_unpack(*H8, V)  # the forward on the values that the backward will see
    L.slora_rmsnorm_fwd_act8(V, g, N, rstd, H8=H8, N8=N8)
    L.slora_rmsnorm_bwd_act8(H8, rstd, g, dN, dX)
    v, gg, dn = R.f64(V), R.f64(g), R.f64(dN)

    def value(h):
        return (h / np.sqrt((h ** 2).mean(1, keepdims=True) + 1e-5) * gg * dn).sum()

    want = np.zeros((T, d))
    for i in np.ndindex(T, d):
        up, dn_ = v.copy(), v.copy()
        up[i] += 1e-4
        dn_[i] -= 1e-4
        want[i] = (value(up) - value(dn_)) / 2e-4
    r = R.f64(rstd)[:, None]
    size = r * np.abs(gg * dn) + np.abs(v) * r ** 3 * np.abs(gg * dn * v).mean(1, keepdims=True)
    assert (np.abs(R.f64(dX) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * size + 1e-6).all()


def test_scratch_of_a_pending_call_is_not_given_to_another_stream(L):
    """A call on the current stream drops its scratch with its kernels pending; calls on a side
    stream at once, without a workspace of their own, must not get that block."""
    T, k, n, r = 256, 512, 384, 16
    gen = gen_of(13)
    W, A, B = rand(gen, (n, k)), rand(gen, (r, k)), rand(gen, (n, r))
    X, XA = rand(gen, (T, k)), rand(gen, (T, r), torch.float32)
    dYs = [rand(gen, (T, n)) for _ in range(2)]
    X8 = L.act8_empty(T, k)
    L.slora_act8_pack(X, *X8)

    def outputs():
        return torch.empty_like(X), torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")

    def call(dY, o, stream=None):
        L.slora_linear_bwd_act8(L.SLICE_NONE, 1, T, [T], k, n, W, A, B, 0.5, None, X8, XA, dY, *o, stream=stream)

    want = [outputs() for _ in dYs]
    for dY, o in zip(dYs, want):
        call(dY, o)
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = [outputs() for _ in dYs]
        torch.cuda.synchronize()
        torch.cuda._sleep(2_000_000)  # about a millisecond in which the first call has not begun
        call(dYs[0], got[0])
        for _ in range(20):           # beside it, from before its start to after its end
            call(dYs[1], got[1], stream=side)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert L.lib().slora_device_error(1) == 0


@pytest.mark.parametrize("side", ["none", "out_rows", "in_cols"])
def test_expired_wait_of_the_sums_is_reported(L, side):
    """With a wait budget of 0 the sums' pipeline gives up (its products' warp cannot find the first
    operand expanded at its first poll): reported and cleared, and the next call is right again."""
    b, s, ctx, k, n, r = 2, 512, [400, 300], 512, 384, 16
    lib = L.lib()
    assert lib.slora_device_error(1) == 0
    cols = {"none": 0, "out_rows": n, "in_cols": k}[side]
    assert lib.slora_set_wait_budget(0) == 0
    try:
        with pytest.raises(AssertionError):  # outputs undefined: dA or dB is off
            linear_case(L, side, b, s, ctx, k, n, r, cols // 2)
        torch.cuda.synchronize()
    finally:
        assert lib.slora_set_wait_budget(-1) == 0
    assert lib.slora_device_error(1) == 7  # SLORA_ERR_TIMEOUT
    assert b"wait expired" in L._lib_err()
    assert lib.slora_device_error(0) == 0
    linear_case(L, side, b, s, ctx, k, n, r, cols // 2)
    assert lib.slora_device_error(0) == 0


@pytest.mark.parametrize("value", [3.4e38, -3.4e38, float("inf"), float("-inf"), float("nan")])
def test_rank_operands_at_the_top_of_fp32(L, value):
    """X A^T and dY B between bf16's and fp32's largest numbers stay finite in the sums' operands, and
    an infinity or NaN reaches its rank column with the formula's signs and no other column."""
    T, k, n, r = 70, 64, 96, 20
    gen = gen_of(17)
    W, A = rand(gen, (n, k)), rand(gen, (r, k))
    X, XA = rand(gen, (T, k)), rand(gen, (T, r), torch.float32)
    X8 = L.act8_empty(T, k)
    L.slora_act8_pack(X, *X8)
    x = R.act8(R.f64(X))[2]
    B = torch.zeros(n, r, device="cuda").bfloat16()
    dY = rand(gen, (T, n), scale=2.0 ** -12)
    dY[:, 0] = 0
    XA[33, 18] = value
    # dY B: row 40 of column 5 is 2^127 + 2^127 (1 - 2^-8), past bf16's largest number; with a value
    # that is not finite, that value
    finite = np.isfinite(value)
    big = np.sign(value) * 2.0 ** 127 * (2 - 2.0 ** -8) if finite else value
    B[0, 5] = 1.0
    if finite:
        B[1, 5] = 1.0
        dY[:, 1] = 0
        dY[40, 0] = dY[40, 1] = float(np.sign(value)) * 2.0 ** 127 * (1 - 2.0 ** -8)
        dY[40, 1] *= 1 + 2.0 ** -7  # 2^127 (1 - 2^-16) rounds to 2^127
        big = float(dY[40, 0].double() + dY[40, 1].double())
        assert 3.3895e38 < abs(big) < 3.4028e38
        X[40] *= 2.0 ** -10  # the sums over tokens stay finite
        L.slora_act8_pack(X, *X8)
        x = R.act8(R.f64(X))[2]
    else:
        dY[40, 0] = value
    dX, dA, dB = torch.empty_like(X), torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")
    L.slora_linear_bwd_act8(L.SLICE_NONE, 1, T, [T], k, n, W, A, B, 0.5, None, X8, XA, dY, dX, dA, dB)
    dy, xa, b = R.f64(dY), R.f64(XA), R.f64(B)
    if not finite:
        # an infinite dY meets zeros of B and the three terms of X A^T: its row of dB, and the
        # columns of dY B that are zero times it, are not finite; column 5 alone is stated
        assert np.isfinite(R.f64(dB)[1:, :18]).all() and np.isfinite(R.f64(dB)[1:, 19]).all()
        col = 0.5 * dy[33, 1:] * value
        got = R.f64(dB)[1:, 18]
        if np.isnan(value):
            assert np.isnan(got).all()
        else:
            assert np.array_equal(got, col)
            assert np.array_equal(R.f64(dA)[5][x[40] != 0], 0.5 * value * x[40][x[40] != 0])
        return
    # (column 18 of dB in rows 0 and 1 overflows by the formula too)
    want = 0.5 * dy.T @ xa
    size = 0.5 * np.abs(dy).T @ np.abs(xa)
    assert (np.abs(R.f64(dB) - want)[2:] <= 1e-5 * size[2:]).all()
    want, size = 0.5 * (dy @ b).T @ x, 0.5 * np.abs(dy @ b).T @ np.abs(x)
    assert (np.abs(R.f64(dA) - want) <= 1e-5 * size).all()


def test_checkpoints_of_no_rows(L):
    d = 64
    X, g = torch.empty(0, d, device="cuda").bfloat16(), torch.ones(d, device="cuda").bfloat16()
    c, c2, rstd = L.act8_empty(0, d), L.act8_empty(0, d), torch.empty(0, device="cuda")
    L.slora_act8_pack(X, *c)
    L.slora_act8_unpack(*c, X)
    L.slora_rmsnorm_fwd_act8(X, g, torch.empty_like(X), rstd, A=X, H=torch.empty_like(X), H8=c, N8=c2)
    L.slora_rmsnorm_bwd_act8(c, rstd, g, X, torch.empty_like(X), dRes=X)
    torch.cuda.synchronize()
    assert L.lib().slora_device_error(1) == 0


@pytest.mark.parametrize("k,n,r", [(256, 688, 16), (136, 72, 64), (64, 520, 5)])
def test_linear_input_gradient_counts_its_roundings(L, k, n, r):
    """dX to its roundings: half a bf16 step of the result, 2^-8 of each term of the LoRA part (whose
    operand lora_scale * dY B is bf16) and 2^-23 of what n + r tensor-core additions add."""
    T, scale = 150, 2.0
    gen = gen_of(n)
    W, A, B = rand(gen, (n, k), scale=k ** -0.5), rand(gen, (r, k), scale=k ** -0.5), rand(gen, (n, r), scale=0.1)
    X, dY, XA = rand(gen, (T, k)), rand(gen, (T, n)), rand(gen, (T, r), torch.float32)
    X8, dX = L.act8_empty(T, k), torch.empty_like(X)
    L.slora_act8_pack(X, *X8)
    dA, dB = torch.empty(r, k, device="cuda"), torch.empty(n, r, device="cuda")
    L.slora_linear_bwd_act8(L.SLICE_NONE, 1, T, [T], k, n, W, A, B, scale, None, X8, XA, dY, dX, dA, dB)
    w, a, dy = R.f64(W), R.f64(A), R.f64(dY)
    p = scale * dy @ R.f64(B)
    want, lora = dy @ w + p @ a, np.abs(p) @ np.abs(a)
    # the operand's own sum over n channels is fp32: n 2^-23 of its terms
    fine = (n + r) * 2.0 ** -23 * (np.abs(dy) @ np.abs(w) + scale * np.abs(dy) @ np.abs(R.f64(B)) @ np.abs(a) + lora)
    assert (np.abs(R.f64(dX) - want) <= 2.0 ** -8 * (np.abs(want) + (1 + 2.0 ** -8) * lora) + (1 + 2.0 ** -8) * fine).all()
