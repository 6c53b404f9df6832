"""Host-side validation of the q/k rotation and of the 8-bit checkpoints: what
the calls refuse, and their workspace queries (no GPU: nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

from tests import qk_reference as R

FAKE = 0x10000  # 16-byte aligned dummy address: never dereferenced
OK, INVALID, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def L():
    from contextual_sparsity_lora_svd_b200 import build
    build.build()
    from contextual_sparsity_lora_svd_b200 import _lib
    return _lib


def status(L, name, args):
    need = ctypes.c_size_t(0)
    return getattr(L.lib(), name)(*args, None, ctypes.byref(need), None), int(need.value)


def dense(L, heads=4, hd=64, **over):
    n = heads * hd
    f = dict(heads=heads, n_idx=0, idx=None, X=FAKE, ldx=n, X_ctx=None, X_out=None, g=FAKE,
             Y=FAKE, ldy=n, dY=FAKE, lddy=n, dX=FAKE * 2, lddx=n, dX_ctx=None, dX_out=None, dg=None)
    f.update(over)
    return L.QkRows(*[f[name] for name, _ in L.QkRows._fields_])


def fwd(L, q, k=None, dt=None, rot=None, hd=64, eps=1e-5, pos=None, ctx=(3, 2)):
    tok, keep = L.make_tokens(2, 5, ctx)
    rot = rot or L.rotary()
    return status(L, "slora_qk_rotary_fwd",
                  [L.BF16 if dt is None else dt, ctypes.byref(tok), hd, eps, ctypes.byref(rot), pos,
                   ctypes.byref(q), None if k is None else ctypes.byref(k)])


def bwd(L, q, k=None, dt=None, gdt=None, hd=64, ctx=(3, 2), **kw):
    tok, keep = L.make_tokens(2, 5, ctx)
    rot = L.rotary()
    dt = L.BF16 if dt is None else dt
    return status(L, "slora_qk_rotary_bwd",
                  [dt, dt if gdt is None else gdt, ctypes.byref(tok), hd, 1e-5, ctypes.byref(rot),
                   None, ctypes.byref(q), None if k is None else ctypes.byref(k)])


def test_dense_calls_need_no_workspace(L):
    assert fwd(L, dense(L), dense(L, 2)) == (OK, 0)
    assert fwd(L, dense(L, g=None), dt=L.F32) == (OK, 0)
    assert bwd(L, dense(L), dense(L, 2)) == (OK, 0)
    st, need = bwd(L, dense(L, dg=FAKE))
    assert st == OK and need >= 64 * 4


def test_sliced_calls(L):
    s = dict(idx=FAKE, n_idx=100, X=None, X_ctx=FAKE, X_out=FAKE, dX_ctx=FAKE, dX_out=FAKE)
    for batch, bytes_ in ((2, 0), (64, 0), (65, 4 * 66)):              # many sequences' offsets
        tok, keep = L.make_tokens(batch, 5, [3] * batch)
        rows, rot = dense(L, **s), L.rotary()
        st, need = status(L, "slora_qk_rotary_fwd", [L.BF16, ctypes.byref(tok), 64, 1e-5, ctypes.byref(rot),
                                                     None, ctypes.byref(rows), None])
        assert st == OK and need >= bytes_ and (need > 0) == (bytes_ > 0)
    assert bwd(L, dense(L, **s))[0] == OK
    assert fwd(L, dense(L, **s), dense(L, 2))[0] == SHAPE              # one sliced, one dense
    assert fwd(L, dense(L, **s), dt=L.F32)[0] == UNSUPPORTED
    assert fwd(L, dense(L, **dict(s, n_idx=257)))[0] == SHAPE
    assert fwd(L, dense(L, **dict(s, n_idx=-1)))[0] == SHAPE
    assert fwd(L, dense(L, **dict(s, X_ctx=None)))[0] == INVALID
    assert fwd(L, dense(L, **dict(s, X_ctx=None)), ctx=(0, 0))[0] == OK  # no context rows
    assert fwd(L, dense(L, **dict(s, X_out=None)), ctx=(5, 5))[0] == OK  # no output rows
    assert bwd(L, dense(L, **dict(s, dX_out=None)))[0] == INVALID
    assert bwd(L, dense(L, **dict(s, X_ctx=None, X_out=None, g=None)))[0] == OK  # x unread


def test_row_refusals(L):
    assert fwd(L, dense(L, X=None))[0] == INVALID
    assert fwd(L, dense(L, Y=None))[0] == INVALID
    assert fwd(L, dense(L, X=FAKE + 8))[0] == ALIGN
    assert fwd(L, dense(L, ldx=255))[0] == SHAPE
    assert fwd(L, dense(L, ldy=255, Y=FAKE * 2))[0] == SHAPE
    assert fwd(L, dense(L, ldy=512))[0] == INVALID                     # in place, another stride
    assert fwd(L, dense(L, heads=0))[0] == SHAPE
    assert fwd(L, dense(L), hd=63)[0] == SHAPE
    assert fwd(L, dense(L), hd=258)[0] == SHAPE
    assert fwd(L, dense(L), eps=0.0)[0] == INVALID
    assert fwd(L, dense(L), eps=float("nan"))[0] == INVALID
    assert fwd(L, dense(L, g=None), eps=0.0)[0] == OK                  # eps unused
    assert fwd(L, dense(L), dt=7)[0] == INVALID
    assert fwd(L, dense(L), pos=FAKE + 2)[0] == ALIGN
    assert fwd(L, dense(L), ctx=(6, 0))[0] == SHAPE
    assert bwd(L, dense(L, dY=None))[0] == INVALID
    assert bwd(L, dense(L, X=None))[0] == INVALID
    assert bwd(L, dense(L, X=None, g=None))[0] == OK
    assert bwd(L, dense(L, dX=FAKE), gdt=L.F32)[0] == INVALID          # dX over a dY of another type
    assert bwd(L, dense(L), dt=L.F32, gdt=L.BF16)[0] == INVALID
    assert bwd(L, dense(L, dg=FAKE + 4))[0] == ALIGN


@pytest.mark.parametrize("kw,want", [
    (dict(dims=66), SHAPE), (dict(dims=3), SHAPE), (dict(dims=-2), SHAPE), (dict(base=1.0), INVALID),
    (dict(base=float("inf")), INVALID), (dict(scaling="linear", factor=0.5), INVALID),
    (dict(scaling="linear", factor=float("nan")), INVALID), (dict(mscale=-1.0), INVALID),
    (dict(scaling="bands", factor=2.0), SHAPE), (dict(scaling="yarn", factor=2.0), SHAPE),
    (dict(scaling="bands", factor=2.0, orig_len=64, low=4.0, high=1.0), INVALID),
    (dict(scaling="ntk", factor=2.0, dims=2), SHAPE),
    (dict(scaling="ntk", factor=1e300, base=1e300, dims=4), INVALID),
    (dict(factor=0.0), OK), (dict(dims=64), OK), (dict(scaling="ntk", factor=2.0), OK)])
def test_rotary_refusals(L, kw, want):
    assert fwd(L, dense(L), rot=L.rotary(**kw))[0] == want
    assert fwd(L, dense(L), rot=L.Rotary(9, 0, 0, 0, 1e4, 1, 0, 0, 0))[0] == INVALID
    assert fwd(L, dense(L), rot=L.Rotary(0, 9, 0, 0, 1e4, 1, 0, 0, 0))[0] == INVALID


def test_binding_refuses_wrong_tensors(L):
    X = torch.zeros(4, 128)
    with pytest.raises(TypeError):
        L.qk_rows(2, X=X, Y=X.bfloat16())
    with pytest.raises(TypeError):
        L.qk_rows(2, X=X, dg=torch.zeros(64, dtype=torch.float64))
    with pytest.raises(TypeError):
        L.qk_rows(2, X_ctx=X, idx=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        L.qk_rows(2, X=X.t())
    with pytest.raises(ValueError):
        L.act8(torch.zeros(4, 100, dtype=torch.int8), torch.zeros(4, 4, dtype=torch.uint8), 4, 100)
    with pytest.raises(TypeError):
        L.slora_qk_rotary_fwd(2, 2, 64, L.qk_rows(2, X=X, Y=X), pos=torch.zeros(4), stream=0)
    with pytest.raises(KeyError):
        L.rotary(scaling="other")


def test_binding_refuses_sizes_that_do_not_fit(L):
    """A tensor too small for the call is refused before any address leaves the binding."""
    bf, f32 = torch.bfloat16, torch.float32
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731
    for rows in (L.qk_rows(2, X=z(3, 128), Y=z(4, 128)), L.qk_rows(2, X=z(4, 64), Y=z(4, 64)),
                 L.qk_rows(2, X=z(4, 128), Y=z(4, 128), g=z(63)),
                 L.qk_rows(2, idx=z(5, dt=torch.int32), X_ctx=z(2, 5), X_out=z(1, 128), Y=z(4, 128)),
                 L.qk_rows(2, idx=z(5, dt=torch.int32), X_ctx=z(2, 4), X_out=z(2, 128), Y=z(4, 128))):
        with pytest.raises(ValueError):
            L.slora_qk_rotary_fwd(2, 2, 64, rows, ctx_len=[1, 1], stream=0)
    with pytest.raises(ValueError):
        L.qk_rows(2)
    H8 = (z(4, 64, dt=torch.int8), z(4, 2, dt=torch.uint8))
    good = dict(X=z(4, 64), g=z(64), N=z(4, 64), rstd=z(4, dt=f32), H8=H8)
    for name, t, err in (("g", z(32), ValueError), ("N", z(3, 64), ValueError), ("N", z(4, 64, dt=f32), TypeError),
                         ("X", z(64, 4).t(), ValueError), ("rstd", z(4), TypeError),
                         ("H8", (H8[0][:3], H8[1]), ValueError)):
        with pytest.raises(err):
            L.slora_rmsnorm_fwd_act8(**dict(good, **{name: t}), stream=0)
    with pytest.raises(ValueError):
        L.slora_rmsnorm_bwd_act8(H8, z(4, dt=f32), z(64), z(4, 64), z(5, 64), stream=0)
    lin = dict(side=L.SLICE_OUT_ROWS, batch=2, seq=2, ctx_len=[1, 1], k=64, n=64, W=z(64, 64), A=z(8, 64),
               B=z(64, 8), lora_scale=1.0, idx=z(16, dt=torch.int32), X8_ctx=H8, XA_save=z(4, 8, dt=f32),
               dY_ctx=z(2, 16), dY_out=z(2, 64), dX_ctx=z(4, 64), dA=z(8, 64, dt=f32), dB=z(64, 8, dt=f32))
    for name, t in (("W", z(64, 32)), ("B", z(8, 8)), ("XA_save", z(2, 8, dt=f32)), ("dY_ctx", z(2, 15)),
                    ("dY_out", z(1, 64)), ("dX_ctx", z(2, 64)), ("dA", z(8, 32, dt=f32))):
        with pytest.raises(ValueError):
            L.slora_linear_bwd_act8(**dict(lin, **{name: t}), stream=0)


def test_act8_refusals(L):
    c = L.Act8(FAKE, FAKE)
    ref = ctypes.byref(c)
    pack = lambda dt, T, d, X, ld, ck: status(L, "slora_act8_pack", [dt, T, d, X, ld, ck])
    assert pack(L.BF16, 4, 100, FAKE, 100, ref) == (OK, 0)
    assert pack(L.F32, 4, 1, FAKE, 1, ref) == (OK, 0)
    assert pack(L.BF16, 0, 100, None, 100, None) == (OK, 0)            # nothing to do
    assert pack(5, 4, 100, FAKE, 100, ref)[0] == INVALID
    assert pack(L.BF16, 4, 0, FAKE, 100, ref)[0] == SHAPE
    assert pack(L.BF16, -1, 8, FAKE, 100, ref)[0] == SHAPE
    assert pack(L.BF16, 4, 100, FAKE, 99, ref)[0] == SHAPE
    assert pack(L.BF16, 4, 100, None, 100, ref)[0] == INVALID
    assert pack(L.BF16, 4, 100, FAKE + 2, 100, ref)[0] == ALIGN
    assert pack(L.BF16, 4, 100, FAKE, 100, None)[0] == INVALID
    half = L.Act8(FAKE, None)
    assert pack(L.BF16, 4, 100, FAKE, 100, ctypes.byref(half))[0] == INVALID
    odd = L.Act8(FAKE, FAKE + 1)
    assert pack(L.BF16, 4, 100, FAKE, 100, ctypes.byref(odd))[0] == ALIGN
    un = lambda T, d, ck, X, ld: status(L, "slora_act8_unpack", [L.BF16, T, d, ck, X, ld])
    assert un(4, 100, ref, FAKE, 100) == (OK, 0)
    assert un(4, 100, None, FAKE, 100)[0] == INVALID
    assert un(4, 100, ref, FAKE, 64)[0] == SHAPE


def test_norm_act8_refusals(L):
    c = L.Act8(FAKE, FAKE)
    ref = ctypes.byref(c)
    f = lambda d=64, A=None, H=None, N=FAKE, h8=ref, n8=ref, dt=L.BF16, eps=1e-5: status(
        L, "slora_rmsnorm_fwd_act8", [dt, 4, d, eps, FAKE, A, FAKE, H, N, FAKE, h8, n8])
    assert f() == (OK, 0)
    assert f(h8=None, n8=None) == (OK, 0)
    assert f(d=16384) == (OK, 0)
    assert f(d=16392)[0] == SHAPE
    assert f(d=60)[0] == SHAPE
    assert f(dt=L.F32)[0] == UNSUPPORTED
    assert f(N=None)[0] == INVALID
    assert f(A=FAKE)[0] == INVALID                                     # H8 of an unstored sum
    assert f(A=FAKE, h8=None) == (OK, 0)
    assert f(eps=-1.0)[0] == INVALID
    b = lambda h8=ref, dN=FAKE, d=64: status(
        L, "slora_rmsnorm_bwd_act8", [L.BF16, 4, d, h8, FAKE, FAKE, dN, None, None, None, FAKE])
    assert b() == (OK, 0)
    assert b(h8=None)[0] == INVALID
    assert b(dN=None)[0] == INVALID
    assert b(d=16392)[0] == SHAPE


def test_linear_bwd_act8_refusals(L):
    tok, keep = L.make_tokens(2, 40, [30, 20])
    c = L.Act8(FAKE, FAKE)
    ref = ctypes.byref(c)

    def call(side, dt=L.BF16, xc=ref, xo=ref, n_idx=20, dyc=FAKE, dyo=FAKE, dxo=FAKE, t=tok, k=72):
        return status(L, "slora_linear_bwd_act8",
                      [dt, ctypes.byref(t), k, 72, FAKE, FAKE, FAKE, 8, 1.0, side, FAKE, n_idx, xc, xo,
                       FAKE, dyc, dyo, FAKE, dxo, FAKE, FAKE])

    for side in (L.SLICE_NONE, L.SLICE_OUT_ROWS, L.SLICE_IN_COLS):
        st, need = call(side)
        assert st == OK and need > 0
        assert call(side, dt=L.F32)[0] == UNSUPPORTED
        assert call(side, xc=None)[0] == INVALID
        assert call(side, dyc=None)[0] == INVALID
        assert call(side, k=70)[0] == SHAPE
    assert call(L.SLICE_IN_COLS, xo=None)[0] == INVALID
    assert call(L.SLICE_IN_COLS, dxo=None)[0] == INVALID
    assert call(L.SLICE_NONE, xo=None, dxo=None)[0] == OK
    assert call(L.SLICE_OUT_ROWS, dyo=None)[0] == INVALID
    assert call(L.SLICE_IN_COLS, n_idx=73)[0] == SHAPE
    none, keep2 = L.make_tokens(2, 40, [0, 0])
    assert call(L.SLICE_IN_COLS, xc=None, t=none)[0] == OK             # no context rows
    assert call(L.SLICE_OUT_ROWS, dyc=None, t=none)[0] == OK


def test_reference_checkpoint_values():
    """The reference itself, on hand-worked blocks."""
    x = np.zeros((1, 40))
    x[0, :3] = [1.0, -0.5, 1.0 / 64]
    x[0, 32] = 3.0
    codes, scales, v = R.act8(x)
    assert codes[0, :3].tolist() == [64, -32, 1] and scales[0].tolist() == [127, 128]
    assert codes[0, 32] == 96 and v[0, 32] == 3.0 and codes[0, 40:].tolist() == [0] * 24
    x[0, 0] = 255.0 / 128  # 127.5 steps: saturates
    assert R.act8(x)[0][0, 0] == 127


def test_reference_frequencies_by_hand():
    f, m = R.frequencies(4, base=100.0)
    assert np.allclose(f, [1.0, 0.1], rtol=1e-15) and m == 1.0
    f, m = R.frequencies(4, base=100.0, scaling="linear", factor=4.0)
    assert np.allclose(f, [0.25, 0.025], rtol=1e-15)
    f, _ = R.frequencies(4, base=100.0, scaling="ntk", factor=10.0)
    assert np.allclose(f, [1.0, 0.01], rtol=1e-12)  # base 100 * 10^2
    # 2 pi / f = 6.28, 62.8 over a context of 31.4: 5 turns and half a turn
    f, _ = R.frequencies(4, base=100.0, scaling="bands", factor=8.0, orig_len=31)
    assert np.allclose(f, [1.0, 0.1 / 8], rtol=1e-15)
    _, m = R.frequencies(8, scaling="yarn", factor=4.0, orig_len=4096)
    assert m == pytest.approx(0.1 * np.log(4.0) + 1.0)


def test_scratch_comes_from_the_pool_of_the_call_s_stream(L, monkeypatch):
    """Scratch that the binding takes for a call on a given stream is allocated with that stream
    current: from another stream's pool it could be a block whose last user still runs."""
    class Stream:
        cuda_stream = 0x40
    current, seen = [None], []

    class Within:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *error):
            current.pop()

    def empty(size, **kw):
        seen.append((size, current[-1]))
        return torch.zeros(size, dtype=torch.uint8)

    class Calls:
        @staticmethod
        def call(*args):  # needs 96 bytes
            ws, size = args[-3], args[-2]._obj
            if ws is None:
                size.value = 96
                return OK
            return OK if size.value >= 96 else WORKSPACE

    monkeypatch.setattr(torch.cuda, "stream", Within)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(L, "_lib", Calls)
    monkeypatch.setattr(L, "_last_need", {})
    st = Stream()
    L._run("call", [], None, st)
    L._run_scratch("call", [], None, st)  # by its query
    L._run_scratch("call", [], None, st)  # by the last call's need
    assert seen == [(96, st)] * 3
    assert L._last_need == {"call": 96} and current == [None]


def test_binding_refuses_tensors_off_the_device(L, monkeypatch):
    """Tensors that fit in type and size but lie on the CPU: their addresses never reach a call."""
    class Calls:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was reached")

    monkeypatch.setattr(L, "_lib", Calls())
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731
    ck = lambda T, d: L.act8_empty(T, d, device="cpu")  # noqa: E731
    X, g = z(4, 128), z(64)
    dense = L.qk_rows(2, X=X, g=g, Y=z(4, 128), dY=z(4, 128), dX=z(4, 128), dg=z(64, dt=f32))
    cut = L.qk_rows(2, g=g, idx=z(8, dt=i32), X_ctx=z(2, 8), X_out=z(2, 128), Y=z(4, 128), dY=z(4, 128),
                    dX_ctx=z(2, 8), dX_out=z(2, 128))
    calls = [lambda f=f, r=r, c=c: f(2, 2, 64, r, ctx_len=c)
             for f in (L.slora_qk_rotary_fwd, L.slora_qk_rotary_bwd) for r, c in ((dense, None), (cut, [1, 1]))]
    calls += [lambda: L.slora_act8_pack(X, *ck(4, 128)), lambda: L.slora_act8_unpack(*ck(4, 128), X),
              lambda: L.slora_rmsnorm_fwd_act8(X, z(128), z(4, 128), H8=ck(4, 128)),
              lambda: L.slora_rmsnorm_bwd_act8(ck(4, 128), z(4, dt=f32), z(128), X, z(4, 128)),
              lambda: L.slora_linear_bwd_act8(
                  L.SLICE_OUT_ROWS, 2, 2, [1, 1], 64, 64, z(64, 64), z(8, 64), z(64, 8), 1.0, z(16, dt=i32),
                  ck(4, 64), z(4, 8, dt=f32), z(2, 16), z(4, 64), z(8, 64, dt=f32), z(64, 8, dt=f32),
                  dY_out=z(2, 64))]
    for call in calls:
        with pytest.raises(ValueError, match="on cpu"):
            call()


def test_binding_refuses_tensors_of_another_device(L, monkeypatch):
    """The same for a tensor of a GPU that is not the current one, and for rows on two devices."""
    class On(torch.Tensor):  # stands in for a tensor of GPU `gpu`
        def get_device(self):
            return self.gpu

    def on(gpu):
        t = torch.zeros(4, 128, dtype=torch.bfloat16).as_subclass(On)
        t.gpu = gpu
        return t

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    L._here(on(1), None, on(1))
    for bad in ([on(0)], [on(1), on(2)], [on(-1)]):
        with pytest.raises(ValueError):
            L._here(*bad)
    assert L.qk_rows(2, X=on(1), Y=on(1)).at == 1
    with pytest.raises(ValueError):
        L.qk_rows(2, X=on(1), Y=on(0))
    rows = L.qk_rows(2, X=on(0), Y=on(0))
    with pytest.raises(ValueError):
        L.slora_qk_rotary_fwd(2, 2, 64, rows)


@pytest.mark.parametrize("which", ["gq", "gk"])
@pytest.mark.parametrize("bad,error", [
    (None, ValueError), (torch.ones(63, dtype=torch.bfloat16), ValueError), (torch.ones(64), TypeError),
    (torch.ones(128, dtype=torch.bfloat16)[::2], ValueError), (torch.ones(64, dtype=torch.bfloat16), ValueError)])
def test_stack_refuses_gains_that_do_not_fit(L, which, bad, error, monkeypatch):
    """A layer without a gain, with a short or strided one or one of another type (and the last: one
    off the device) is refused before anything is allocated."""
    from contextual_sparsity_lora_svd_b200 import layers

    def nothing(*a, **k):
        raise AssertionError("allocated")

    good = torch.ones(64, dtype=torch.bfloat16)
    lays = [dict(gq=good, gk=good), dict(gq=good, gk=good)]
    lays[1][which] = bad
    if bad is None:
        del lays[1][which]
    here = L._here
    monkeypatch.setattr(L, "_here", lambda t: None if t is good else here(t))
    monkeypatch.setattr(torch, "empty", nothing)
    with pytest.raises(error):
        layers.DecoderStack(lays, 256, 4, 2, 64, 688, 8, 8, 1.0, 1, 8, [8], [0.0] * 2, [0.0] * 2, None, None,
                            qk_norm=True)


def test_a_gain_s_gradient_needs_the_gain(L):
    """dg without g would never be written: refused, of either tensor."""
    assert bwd(L, dense(L, g=None, dg=FAKE))[0] == INVALID
    assert bwd(L, dense(L), dense(L, 2, g=None, dg=FAKE))[0] == INVALID
    assert bwd(L, dense(L, dg=FAKE), dense(L, 2, g=None))[0] == OK


def test_norms_of_no_rows(L):
    """Tensors without rows have no address; there is nothing to do, as in slora_act8_pack."""
    assert status(L, "slora_rmsnorm_fwd_act8",
                  [L.BF16, 0, 64, 1e-5, None, None, FAKE, None, None, None, None, None]) == (OK, 0)
    assert status(L, "slora_rmsnorm_bwd_act8",
                  [L.BF16, 0, 64, None, None, FAKE, None, None, None, None, None]) == (OK, 0)
    none = L.Act8(None, None)
    assert status(L, "slora_rmsnorm_fwd_act8", [L.BF16, 0, 64, 1e-5, None, None, FAKE, None, None, None,
                                                ctypes.byref(none), ctypes.byref(none)]) == (OK, 0)
    assert status(L, "slora_rmsnorm_fwd_act8",
                  [L.BF16, 0, 60, 1e-5, None, None, FAKE, None, None, None, None, None])[0] == SHAPE


@pytest.mark.parametrize("ctx", [[3], [3, 2, 1], []])
def test_binding_refuses_context_lengths_of_another_batch(L, ctx):
    """A sequence without a length is no sequence without context rows."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    tc = sum(ctx)
    rows = L.qk_rows(2, idx=z(5, dt=torch.int32), X_ctx=z(tc, 5), X_out=z(10 - tc, 128), Y=z(10, 128))
    with pytest.raises(ValueError, match="context lengths for 2 sequences"):
        L.slora_qk_rotary_fwd(2, 5, 64, rows, ctx_len=ctx)
    f32 = torch.float32
    with pytest.raises(ValueError, match="context lengths for 2 sequences"):
        L.slora_linear_bwd_act8(L.SLICE_OUT_ROWS, 2, 5, ctx, 64, 64, z(64, 64), z(8, 64), z(64, 8), 1.0,
                                z(16, dt=torch.int32), L.act8_empty(10, 64, device="cpu"), z(10, 8, dt=f32),
                                z(tc, 16), z(10, 64), z(8, 64, dt=f32), z(64, 8, dt=f32), dY_out=z(10 - tc, 64))
