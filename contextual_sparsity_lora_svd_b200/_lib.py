"""ctypes binding of libslora.so (the C ABI in include/slora.h).

Argument marshalling only: each function takes torch tensors (device memory
owned by the caller) or raw integer pointers, passes their addresses to the C
call of the same name on the current CUDA stream, and raises SloraError on a
non-zero status.  Workspace is taken from a caller tensor or, when omitted,
allocated once per call with torch (plumbing, not compute).  Nothing here
computes any part of the method; a missing library raises at import time.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libslora.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m contextual_sparsity_lora_svd_b200.build` "
        "(the CUDA library is required; there is no fallback)")
_lib = ctypes.CDLL(LIB_PATH)

c_int, c_i32, c_i64, c_u64, c_f32, c_vp, c_sz = (ctypes.c_int, ctypes.c_int32, ctypes.c_int64,
                                                  ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p,
                                                  ctypes.c_size_t)
P_SZ = ctypes.POINTER(c_sz)
P_I32 = ctypes.POINTER(c_i32)

F32, BF16 = 0, 1
CRIT_FFN, CRIT_QK, CRIT_FFN_GRAM, CRIT_QK_ROPE_PAIR, CRIT_L2 = 0, 1, 2, 3, 4
SLICE_NONE, SLICE_OUT_ROWS, SLICE_IN_COLS = 0, 1, 2

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "SHAPE", 3: "ALIGN", 4: "WORKSPACE", 5: "UNSUPPORTED",
          6: "CUDA", 7: "TIMEOUT"}


class SloraError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({status}): {msg}")
        self.status = status


class Tokens(ctypes.Structure):
    _fields_ = [("batch", c_i32), ("seq", c_i32), ("ctx_len", P_I32)]


class FfnLayer(ctypes.Structure):
    _fields_ = [("d", c_i64), ("d_ff", c_i64), ("r_svd", c_i32), ("r_lora", c_i32),
                ("lora_scale", c_f32),
                ("Wg", c_vp), ("Wu", c_vp), ("Wd_t", c_vp),
                ("Ag", c_vp), ("Bg", c_vp), ("Au", c_vp), ("Bu", c_vp), ("Ad", c_vp), ("Bd", c_vp),
                ("Lg", c_vp), ("Ug", c_vp), ("Lu", c_vp), ("Uu", c_vp)]


class FfnGrads(ctypes.Structure):
    _fields_ = [("dAg", c_vp), ("dBg", c_vp), ("dAu", c_vp), ("dBu", c_vp), ("dAd", c_vp),
                ("dBd", c_vp)]


class Rotary(ctypes.Structure):
    _fields_ = [("layout", c_i32), ("scaling", c_i32), ("dims", c_i32), ("orig_len", c_i32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("mscale", ctypes.c_double)]


class QkRows(ctypes.Structure):
    _fields_ = [("heads", c_i32), ("n_idx", c_i32), ("idx", c_vp), ("X", c_vp), ("ldx", c_i64),
                ("X_ctx", c_vp), ("X_out", c_vp), ("g", c_vp), ("Y", c_vp), ("ldy", c_i64),
                ("dY", c_vp), ("lddy", c_i64), ("dX", c_vp), ("lddx", c_i64), ("dX_ctx", c_vp),
                ("dX_out", c_vp), ("dg", c_vp)]


class Act8(ctypes.Structure):
    _fields_ = [("codes", c_vp), ("scales", c_vp)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_lib_err = _sig("slora_last_error_string", ctypes.c_char_p, [])
_sig("slora_version", c_int, [])
_sig("slora_device_error", c_int, [c_int])
_sig("slora_set_wait_budget", c_int, [c_i64])
_sig("slora_svd_prepare", c_int,
     [c_vp, c_i64, c_i64, c_int, c_int, c_int, c_u64, c_vp, c_vp, c_vp, c_vp, P_SZ, c_vp])
_sig("slora_estimate_select", c_int,
     [c_int, c_vp, c_int, ctypes.POINTER(Tokens), c_i64, c_vp, c_vp, c_i64, c_vp, c_vp, c_i64,
      c_int, c_int, c_int, c_int, ctypes.c_double, c_vp, P_I32, c_vp, c_vp, P_SZ, c_vp])
_LIN = [c_int, ctypes.POINTER(Tokens), c_i64, c_i64, c_vp, c_vp, c_vp, c_int, c_f32, c_int, c_vp,
        c_i32]
_sig("slora_linear_fwd", c_int, _LIN + [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_SZ, c_vp])
_sig("slora_linear_bwd", c_int,
     _LIN + [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_SZ, c_vp])
_sig("slora_ffn_fwd_bwd", c_int,
     [c_int, ctypes.POINTER(FfnLayer), ctypes.POINTER(Tokens), ctypes.c_double, c_vp, c_vp, c_vp,
      c_vp,
      ctypes.POINTER(FfnGrads), c_vp, P_I32, c_vp, c_i32, c_vp, P_SZ, c_vp])

_sig("slora_ffn_bwd", c_int,
     [c_int, ctypes.POINTER(FfnLayer), ctypes.POINTER(Tokens), ctypes.c_double, c_vp, c_vp, c_vp,
      c_vp, ctypes.POINTER(FfnGrads), c_vp, P_I32, c_vp, c_i32, c_vp, P_SZ, c_vp])
_sig("slora_ffn_fwd_bwd_per_seq", c_int,
     [c_int, ctypes.POINTER(FfnLayer), ctypes.POINTER(Tokens), ctypes.c_double, c_vp, c_vp, c_vp,
      c_vp, ctypes.POINTER(FfnGrads), c_vp, P_I32, c_vp, c_i32, c_vp, P_SZ, c_vp])
_sig("slora_rope_pack", c_int,
     [c_int, ctypes.POINTER(Tokens), c_i64, c_int, ctypes.c_double, c_vp, c_i32, c_vp, c_vp, c_vp,
      c_vp, c_vp, P_SZ, c_vp])
_sig("slora_rope_unpack", c_int,
     [c_int, ctypes.POINTER(Tokens), c_i64, c_int, ctypes.c_double, c_vp, c_i32, c_vp, c_vp, c_vp,
      c_vp, c_vp, P_SZ, c_vp])
_sig("slora_attention_fwd", c_int,
     [c_int, ctypes.POINTER(Tokens), c_int, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_SZ,
      c_vp])
_sig("slora_attention_bwd", c_int,
     [c_int, ctypes.POINTER(Tokens), c_int, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
      c_vp, c_vp, c_vp, P_SZ, c_vp])
_sig("slora_rmsnorm_fwd", c_int,
     [c_int, c_i64, c_i64, c_f32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_SZ, c_vp])
_sig("slora_rmsnorm_bwd", c_int,
     [c_int, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_SZ, c_vp])

_QK = [ctypes.POINTER(Tokens), c_int, c_f32, ctypes.POINTER(Rotary), c_vp, ctypes.POINTER(QkRows),
       ctypes.POINTER(QkRows), c_vp, P_SZ, c_vp]
_sig("slora_qk_rotary_fwd", c_int, [c_int] + _QK)
_sig("slora_qk_rotary_bwd", c_int, [c_int, c_int] + _QK)
P_ACT8 = ctypes.POINTER(Act8)
_sig("slora_act8_pack", c_int, [c_int, c_i64, c_i64, c_vp, c_i64, P_ACT8, c_vp, P_SZ, c_vp])
_sig("slora_act8_unpack", c_int, [c_int, c_i64, c_i64, P_ACT8, c_vp, c_i64, c_vp, P_SZ, c_vp])
_sig("slora_rmsnorm_fwd_act8", c_int,
     [c_int, c_i64, c_i64, c_f32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_ACT8, P_ACT8, c_vp, P_SZ,
      c_vp])
_sig("slora_rmsnorm_bwd_act8", c_int,
     [c_int, c_i64, c_i64, P_ACT8, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_SZ, c_vp])
_sig("slora_linear_bwd_act8", c_int,
     _LIN + [P_ACT8, P_ACT8, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, P_SZ, c_vp])

_sig("slora_noalloc_scratch_bytes", c_sz, [])
_sig("slora_estimate_select_noalloc", c_int,
     [c_int, c_vp, c_int, ctypes.POINTER(Tokens), c_i64, c_vp, c_vp, c_i64, c_vp, c_vp, c_i64,
      c_int, c_int, c_int, c_int, ctypes.c_double, c_vp, P_I32, c_vp, c_vp])
_sig("slora_launch_count", c_i64, [])
_sig("slora_profile_enable", None, [c_int])
_sig("slora_profile_read", c_int, [ctypes.c_char_p, ctypes.POINTER(c_i64),
                                   ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)])

EXPORTS = sorted(["slora_last_error_string", "slora_version", "slora_svd_prepare",
                  "slora_estimate_select", "slora_linear_fwd", "slora_linear_bwd",
                  "slora_ffn_fwd_bwd", "slora_launch_count", "slora_profile_enable",
                  "slora_profile_read", "slora_noalloc_scratch_bytes",
                  "slora_estimate_select_noalloc", "slora_device_error",
                  "slora_set_wait_budget", "slora_ffn_bwd", "slora_ffn_fwd_bwd_per_seq",
                  "slora_rope_pack", "slora_rope_unpack",
                  "slora_attention_fwd", "slora_attention_bwd", "slora_rmsnorm_fwd",
                  "slora_rmsnorm_bwd", "slora_qk_rotary_fwd", "slora_qk_rotary_bwd",
                  "slora_act8_pack", "slora_act8_unpack", "slora_rmsnorm_fwd_act8",
                  "slora_rmsnorm_bwd_act8", "slora_linear_bwd_act8"])


def lib():
    return _lib


def version() -> int:
    return _lib.slora_version()


def launch_count() -> int:
    return int(_lib.slora_launch_count())


def profile_enable(on: bool) -> None:
    _lib.slora_profile_enable(1 if on else 0)


def profile_read(kernel_class: str) -> tuple[int, float, float]:
    """(launches, total_ms, work) recorded for a kernel class since enabling."""
    n, ms, w = c_i64(0), ctypes.c_double(0), ctypes.c_double(0)
    _check("slora_profile_read", _lib.slora_profile_read(kernel_class.encode(), ctypes.byref(n),
                                                         ctypes.byref(ms), ctypes.byref(w)))
    return int(n.value), float(ms.value), float(w.value)


KERNEL_CLASSES = ["gemm_tc", "gemm_simt", "estimate", "select", "elementwise", "aux", "prepare",
                  "skinny", "compact", "attention", "norm"]


def ptr(x) -> int | None:
    """Device address of a tensor (None/0 -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x or None
    return x.data_ptr() or None


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> int | None:
    if stream is None:  # the handle alone: torch.cuda.current_stream() takes 6 us to wrap it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) or None
    return stream.cuda_stream or None


def _check(fn, st):
    if st != 0:
        raise SloraError(fn, st, _lib_err().decode())


def make_tokens(batch: int, seq: int, ctx_len) -> tuple[Tokens, object]:
    """ctypes token struct; returns (struct, keep-alive host array)."""
    arr = (c_i32 * batch)(*[int(c) for c in ctx_len])
    return Tokens(batch, seq, ctypes.cast(arr, P_I32)), arr


def _scratch(size, stream):
    """Device bytes for a call on `stream` (None: the current one), from that stream's own pool.
    A block of another stream's pool may still be in use there; and this one, dropped with the
    call pending, goes to later work of the same stream alone."""
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device="cuda")


def _run(fn_name, args_before_ws, ws, stream):
    """Query the workspace size, take/allocate it, run the call."""
    f = getattr(_lib, fn_name)
    need, st = c_sz(0), _stream(stream)
    _check(fn_name, f(*args_before_ws, None, ctypes.byref(need), st))
    owned = None
    if ws is None:
        owned = _scratch(max(int(need.value), 16), stream)
        ws = owned
    have = c_sz(ws.numel() * ws.element_size())
    _check(fn_name, f(*args_before_ws, ptr(ws), ctypes.byref(have), st))
    return owned


def workspace_size(fn_name, args_before_ws) -> int:
    f = getattr(_lib, fn_name)
    need = c_sz(0)
    _check(fn_name, f(*args_before_ws, None, ctypes.byref(need), None))
    return int(need.value)


# ------------------------------------------------------------------ calls
def slora_svd_prepare(W, rank, L, U, W_t=None, n_iter=0, seed=0, ws=None, stream=None):
    n, k = W.shape
    return _run("slora_svd_prepare",
                [ptr(W), n, k, dtype_code(W), rank, n_iter, seed, ptr(L), ptr(U), ptr(W_t)],
                ws, stream)


def slora_estimate_select(crit, X, batch, seq, ctx_len, L0, U0, L1, U1, rank, sparsity, idx_out,
                          heads=0, kv_heads=0, head_dim=0, scores_out=None, ws=None, stream=None):
    """Returns k_keep (FFN) or k_h (QK)."""
    tok, keep = make_tokens(batch, seq, ctx_len)
    k_out = c_i32(0)
    _run("slora_estimate_select",
         [crit, ptr(X), dtype_code(X), ctypes.byref(tok), X.shape[1], ptr(L0), ptr(U0),
          U0.shape[0], ptr(L1), ptr(U1), U1.shape[0], rank, heads, kv_heads, head_dim,
          float(sparsity), ptr(idx_out), ctypes.byref(k_out), ptr(scores_out)], ws, stream)
    del keep
    return int(k_out.value)


def slora_estimate_select_noalloc(crit, X, batch, seq, ctx_len, L0, U0, L1, U1, rank, sparsity,
                                  idx_out, heads=0, kv_heads=0, head_dim=0, scores_out=None,
                                  stream=None):
    """slora_estimate_select with the library's built-in scratch buffer (no
    workspace argument, nothing allocated).  Returns k_keep (FFN) or k_h (QK)."""
    tok, keep = make_tokens(batch, seq, ctx_len)
    k_out = c_i32(0)
    _check("slora_estimate_select_noalloc", _lib.slora_estimate_select_noalloc(
        crit, ptr(X), dtype_code(X), ctypes.byref(tok), X.shape[1], ptr(L0), ptr(U0),
        U0.shape[0], ptr(L1), ptr(U1), U1.shape[0], rank, heads, kv_heads, head_dim,
        float(sparsity), ptr(idx_out), ctypes.byref(k_out), ptr(scores_out), _stream(stream)))
    del keep
    return int(k_out.value)


def noalloc_scratch_bytes() -> int:
    return int(_lib.slora_noalloc_scratch_bytes())


def slora_linear_fwd(side, batch, seq, ctx_len, k, n, W, A, B, lora_scale, idx, X_ctx,
                     Y_ctx, X_out=None, Y_out=None, XA_save=None, ws=None, stream=None):
    tok, keep = make_tokens(batch, seq, ctx_len)
    n_idx = 0 if idx is None else idx.numel()
    _run("slora_linear_fwd",
         [dtype_code(W), ctypes.byref(tok), k, n, ptr(W), ptr(A), ptr(B), A.shape[0],
          float(lora_scale), side, ptr(idx), n_idx, ptr(X_ctx), ptr(X_out), ptr(Y_ctx),
          ptr(Y_out), ptr(XA_save)], ws, stream)
    del keep


def slora_linear_bwd(side, batch, seq, ctx_len, k, n, W, A, B, lora_scale, idx, X_ctx, XA_save,
                     dY_ctx, dX_ctx, dA, dB, X_out=None, dY_out=None, dX_out=None, ws=None,
                     stream=None):
    tok, keep = make_tokens(batch, seq, ctx_len)
    n_idx = 0 if idx is None else idx.numel()
    _run("slora_linear_bwd",
         [dtype_code(W), ctypes.byref(tok), k, n, ptr(W), ptr(A), ptr(B), A.shape[0],
          float(lora_scale), side, ptr(idx), n_idx, ptr(X_ctx), ptr(X_out), ptr(XA_save),
          ptr(dY_ctx), ptr(dY_out), ptr(dX_ctx), ptr(dX_out), ptr(dA), ptr(dB)], ws, stream)
    del keep


def ffn_layer_struct(d, d_ff, r_svd, r_lora, lora_scale, Wg, Wu, Wd_t, Ag, Bg, Au, Bu, Ad, Bd,
                     Lg=None, Ug=None, Lu=None, Uu=None) -> FfnLayer:
    return FfnLayer(d, d_ff, r_svd, r_lora, float(lora_scale), ptr(Wg), ptr(Wu), ptr(Wd_t),
                    ptr(Ag), ptr(Bg), ptr(Au), ptr(Bu), ptr(Ad), ptr(Bd), ptr(Lg), ptr(Ug),
                    ptr(Lu), ptr(Uu))


def ffn_grads_struct(dAg, dBg, dAu, dBu, dAd, dBd) -> FfnGrads:
    return FfnGrads(ptr(dAg), ptr(dBg), ptr(dAu), ptr(dBu), ptr(dAd), ptr(dBd))


def ffn_args(dt, layer, batch, seq, ctx_len, sparsity, X, dOut, out, dX, grads, idx_out,
             idx_force=None):
    """Positional arguments of slora_ffn_fwd_bwd before (ws, ws_bytes, stream)
    plus the objects that must stay alive while they are used."""
    tok, keep = make_tokens(batch, seq, ctx_len)
    k_out = c_i32(0)
    k_force = 0 if idx_force is None else idx_force.numel()
    args = [dt, ctypes.byref(layer), ctypes.byref(tok), float(sparsity), ptr(X), ptr(dOut),
            ptr(out), ptr(dX), None if grads is None else ctypes.byref(grads), ptr(idx_out),
            ctypes.byref(k_out),
            ptr(idx_force), k_force]
    return args, (tok, keep, k_out, layer, grads)


def slora_ffn_fwd_bwd(layer: FfnLayer, batch, seq, ctx_len, sparsity, X, dOut, out, dX,
                      grads: FfnGrads, idx_out, idx_force=None, ws=None, stream=None,
                      per_sequence=False) -> int:
    """Returns k_keep.  per_sequence: one channel set per sequence
    (slora_ffn_fwd_bwd_per_seq; idx_out is [batch x d_ff], idx_force
    [batch x k_force])."""
    args, keep = ffn_args(dtype_code(X), layer, batch, seq, ctx_len, sparsity, X, dOut, out, dX,
                          grads, idx_out, idx_force)
    if per_sequence and idx_force is not None:
        args[-1] = idx_force.numel() // batch
    _run("slora_ffn_fwd_bwd_per_seq" if per_sequence else "slora_ffn_fwd_bwd", args, ws, stream)
    return int(keep[2].value)


def slora_ffn_bwd(layer: FfnLayer, batch, seq, ctx_len, sparsity, X, dOut, out, dX,
                  grads: FfnGrads, idx_out, ws, idx_force=None, stream=None) -> int:
    """The backward half on the workspace `ws` of an earlier forward-only
    slora_ffn_fwd_bwd call with the same arguments.  Returns k_keep."""
    args, keep = ffn_args(dtype_code(X), layer, batch, seq, ctx_len, sparsity, X, dOut, out, dX,
                          grads, idx_out, idx_force)
    _run("slora_ffn_bwd", args, ws, stream)
    return int(keep[2].value)


def ffn_workspace_bytes(layer: FfnLayer, batch, seq, ctx_len, sparsity, X, out, idx_out,
                        idx_force=None) -> int:
    args, keep = ffn_args(dtype_code(X), layer, batch, seq, ctx_len, sparsity, X, None, out, None,
                          None, idx_out, idx_force)
    return workspace_size("slora_ffn_fwd_bwd", args)


# ------------------------------------------- decoder-layer pieces
ROPE_BASE = 10000.0
RMS_EPS = 1e-5


def slora_rope_pack(batch, seq, ctx_len, n, head_dim, Y_rot, Y=None, Y_ctx=None, Y_out=None,
                    idx=None, rope_base=ROPE_BASE, ws=None, stream=None):
    tok, keep = make_tokens(batch, seq, ctx_len)
    n_idx = 0 if idx is None else idx.numel()
    _run("slora_rope_pack", [BF16, ctypes.byref(tok), n, head_dim, float(rope_base), ptr(idx),
                             n_idx, ptr(Y), ptr(Y_ctx), ptr(Y_out), ptr(Y_rot)], ws, stream)
    del keep


def slora_rope_unpack(batch, seq, ctx_len, n, head_dim, G, dY=None, dY_ctx=None, dY_out=None,
                      idx=None, rope_base=ROPE_BASE, ws=None, stream=None):
    tok, keep = make_tokens(batch, seq, ctx_len)
    n_idx = 0 if idx is None else idx.numel()
    _run("slora_rope_unpack", [BF16, ctypes.byref(tok), n, head_dim, float(rope_base), ptr(idx),
                               n_idx, ptr(G), ptr(dY), ptr(dY_ctx), ptr(dY_out)], ws, stream)
    del keep


def slora_attention_fwd(batch, seq, heads, kv_heads, head_dim, Q, K, V, O, lse, stream=None):
    tok, keep = make_tokens(batch, seq, [seq] * batch)
    _run("slora_attention_fwd", [BF16, ctypes.byref(tok), heads, kv_heads, head_dim, ptr(Q),
                                 ptr(K), ptr(V), ptr(O), ptr(lse)], None, stream)
    del keep


def slora_attention_bwd(batch, seq, heads, kv_heads, head_dim, Q, K, V, O, lse, dO, dQ, dK, dV,
                        ws=None, stream=None):
    tok, keep = make_tokens(batch, seq, [seq] * batch)
    _run("slora_attention_bwd", [BF16, ctypes.byref(tok), heads, kv_heads, head_dim, ptr(Q),
                                 ptr(K), ptr(V), ptr(O), ptr(lse), ptr(dO), ptr(dQ), ptr(dK),
                                 ptr(dV)], ws, stream)
    del keep


def slora_rmsnorm_fwd(X, g, N=None, A=None, H=None, rstd=None, eps=RMS_EPS, stream=None):
    T, d = X.shape
    _run("slora_rmsnorm_fwd", [BF16, T, d, float(eps), ptr(X), ptr(A), ptr(g), ptr(H), ptr(N),
                               ptr(rstd)], None, stream)


def slora_rmsnorm_bwd(H, rstd, g, dN0, dX, dN1=None, dN2=None, dRes=None, stream=None):
    T, d = H.shape
    _run("slora_rmsnorm_bwd", [BF16, T, d, ptr(H), ptr(rstd), ptr(g), ptr(dN0), ptr(dN1),
                               ptr(dN2), ptr(dRes), ptr(dX)], None, stream)


# ------------------------------------- rotation of q and k with head norms
ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


@functools.lru_cache(maxsize=64)
def rotary(layout="half", dims=0, base=ROPE_BASE, scaling="none", factor=1.0, orig_len=0, low=0.0,
           high=0.0, mscale=0.0) -> Rotary:
    """How q and k are rotated (slora_rotary); dims 0: the whole head.  Equal
    arguments give the same struct: it is not to be changed."""
    return Rotary(ROTARY_LAYOUTS[layout], ROTARY_SCALINGS[scaling], int(dims), int(orig_len),
                  float(base), float(factor), float(low), float(high), float(mscale))


def _rows(t, what):
    """(address, row stride) of a 2-D tensor whose rows are contiguous."""
    st = t.stride()
    if len(st) == 2 and st[1] == 1 and st[0] > 1:
        return t.data_ptr(), st[0]
    n = t.shape
    if len(st) != 2 or (st[1] != 1 and n[1] > 1):
        raise ValueError(f"{what}: a 2-D tensor with contiguous rows is needed")
    return t.data_ptr(), st[0] if n[0] > 1 else max(st[0], n[1])


def _whole(t, what, dt, at):
    if t.dtype is not dt:
        raise TypeError(f"{what} is {t.dtype}, not {dt}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous tensor is needed")
    if t.get_device() != at:
        raise ValueError(f"{what} is on {t.device}, not where the rows are")
    return t.data_ptr()


def _same(t, what, dt, at):
    if t.dtype != dt:
        raise TypeError(f"{what} is {t.dtype}, the rows are {dt}")
    if t.get_device() != at:
        raise ValueError(f"{what} is on {t.device}, not where the rows are")


def _here(*tensors):
    """Refuses tensors (None stays None) that are not on the current CUDA device."""
    at = None
    for t in tensors:
        if t is not None:
            d = t.get_device()  # -1: on the CPU
            if d != at:
                if at is not None or d < 0 or d != torch._C._cuda_getDevice():
                    raise ValueError(f"a tensor on {t.device} is no operand of a call on the current CUDA device")
                at = d


def _fit(t, what, n, dt):
    """Address of a contiguous tensor of n elements (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dt:
        raise TypeError(f"{what} is {t.dtype}, not {dt}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous tensor of {n} elements is needed")
    return t.data_ptr() or None


def qk_rows(heads, X=None, g=None, Y=None, dY=None, dX=None, dg=None, idx=None, X_ctx=None,
            X_out=None, dX_ctx=None, dX_out=None) -> QkRows:
    """The rows of q or k for slora_qk_rotary_fwd / _bwd: dense (X, Y, dX may
    have any row stride), or with `idx` sliced (X_ctx, X_out, dX_ctx, dX_out
    contiguous).  The struct keeps its tensors alive; a program that calls more
    than once on the same buffers builds it once."""
    r = QkRows(heads)
    first = X if X is not None else Y if Y is not None else dX
    if first is None:
        first = next((t for t in (X_ctx, X_out, dX_ctx, dX_out, dY) if t is not None), None)
        if first is None:
            raise ValueError("rows without a tensor")
    dt, at = first.dtype, first.get_device()
    r.at = at
    r.dt = _DTYPES.get(dt)
    if r.dt is None:
        raise TypeError("the rows are bf16 or fp32 tensors")
    if X is not None:
        r.X, r.ldx = _rows(X, "X")
    if Y is not None:
        if Y is X:
            r.Y, r.ldy = r.X, r.ldx
        else:
            r.Y, r.ldy = _rows(Y, "Y")
            _same(Y, "Y", dt, at)
    if dX is not None:
        r.dX, r.lddx = _rows(dX, "dX")
        _same(dX, "dX", dt, at)
    if g is not None:
        r.g = _whole(g, "g", dt, at)
    r.gdt = F32
    if dY is not None:
        r.dY, r.lddy = _rows(dY, "dY")
        r.gdt = dtype_code(dY)
        _same(dY, "dY", dY.dtype, at)
    if dg is not None:
        r.dg = _whole(dg, "dg", torch.float32, at)
    if idx is not None:
        r.n_idx = idx.numel()
        if X_ctx is not None:
            r.X_ctx = _whole(X_ctx, "X_ctx", dt, at)
        if X_out is not None:
            r.X_out = _whole(X_out, "X_out", dt, at)
        if dX_ctx is not None:
            r.dX_ctx = _whole(dX_ctx, "dX_ctx", dt, at)
        if dX_out is not None:
            r.dX_out = _whole(dX_out, "dX_out", dt, at)
        # an empty list is still a list: its address, never read, may be null
        r.idx = _whole(idx, "idx", torch.int32, at) or r.X_out or r.dX_out or r.Y or r.dY
    r.tensors = (X, g, Y, dY, dX, dg, idx, X_ctx, X_out, dX_ctx, dX_out)
    return r


_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


@functools.lru_cache(maxsize=64)
def _tokens(batch, seq, ctx_len):
    """(struct, its host array, context rows); ctx_len a tuple, or None: undivided."""
    if ctx_len is None:
        ctx_len = (seq,) * batch
    if len(ctx_len) != batch:
        raise ValueError(f"{len(ctx_len)} context lengths for {batch} sequences")
    return *make_tokens(batch, seq, ctx_len), sum(ctx_len)


def _sizes(r, T, TC, head_dim):
    """Refuses tensors of a qk_rows that do not hold T rows of its heads."""
    n = r.heads * head_dim
    X, g, Y, dY, dX, dg, idx, X_ctx, X_out, dX_ctx, dX_out = r.tensors
    shape = (T, n)
    for t in (X, None if Y is X else Y, dY, None if dX is dY else dX):
        if t is not None and t.shape != shape:
            raise ValueError(f"rows of {T} x {n} are needed, not {tuple(t.shape)}")
    if g is not None or dg is not None:
        for t in (g, dg):
            if t is not None and t.numel() != head_dim:
                raise ValueError(f"g and dg have one value a channel of a head, {head_dim}")
    if idx is not None:
        for t, want in ((X_ctx, TC * r.n_idx), (dX_ctx, TC * r.n_idx), (X_out, (T - TC) * n),
                        (dX_out, (T - TC) * n)):
            if t is not None and t.numel() != want:
                raise ValueError(f"sliced rows: {want} elements are needed, not {t.numel()}")


def _qk(fn, head, batch, seq, head_dim, q, k, rotary_, pos, eps, ctx_len, ws, stream):
    tok, keep, TC = _tokens(batch, seq, None if ctx_len is None else tuple(map(int, ctx_len)))
    if pos is not None and (pos.dtype != torch.int32 or pos.numel() != batch * seq
                            or not pos.is_contiguous()):
        raise TypeError("pos is a contiguous int32 tensor with one position a row")
    kr = None
    if k is not None:
        if k.dt != q.dt or k.gdt != q.gdt:
            raise TypeError("q and k have the same dtypes")
        kr = ctypes.byref(k)
    _sizes(q, batch * seq, TC, head_dim)
    if k is not None:
        _sizes(k, batch * seq, TC, head_dim)
    at = q.at  # where each of a qk_rows' tensors is
    if (at < 0 or at != torch._C._cuda_getDevice() or (k is not None and k.at != at)
            or (pos is not None and pos.get_device() != at) or ws is not None):
        _here(*q.tensors, *(() if k is None else k.tensors), pos, ws)
    args = head + [ctypes.byref(tok), head_dim, eps, ctypes.byref(rotary_ or rotary()), ptr(pos),
                   ctypes.byref(q), kr]
    _run_scratch(fn, args, ws, stream)
    del keep


_NO_BYTES = ctypes.byref(c_sz(0))  # written by workspace queries alone
_last_need = {}  # bytes that a function's last call took
_SMALL = 1 << 20


def _run_plain(fn_name, args, stream):
    """A call that needs no scratch: any non-null workspace address runs it."""
    st = getattr(_lib, fn_name)(*args, 16, _NO_BYTES, _stream(stream))
    if st:
        _check(fn_name, st)


def _run_scratch(fn_name, args, ws, stream):
    """_run without its query where the scratch of the last such call does (a call
    with too little starts nothing); large scratch is asked for each time."""
    if ws is not None:
        size = ws.numel() * ws.element_size()
        _check(fn_name, getattr(_lib, fn_name)(*args, ptr(ws), ctypes.byref(c_sz(size)),
                                               _stream(stream)))
        return
    size = _last_need.get(fn_name, 0)
    if size <= _SMALL:
        if size:
            ws = _scratch(size, stream)
            st = getattr(_lib, fn_name)(*args, ws.data_ptr(), ctypes.byref(c_sz(size)),
                                        _stream(stream))
        else:
            st = getattr(_lib, fn_name)(*args, 16, _NO_BYTES, _stream(stream))
        if st != 4:  # SLORA_ERR_WORKSPACE
            _check(fn_name, st)
            return
    _last_need[fn_name] = _run(fn_name, args, None, stream).numel()


def slora_qk_rotary_fwd(batch, seq, head_dim, q, k=None, rotary=None, pos=None, eps=RMS_EPS,
                        ctx_len=None, ws=None, stream=None):
    """Rotates (and, with a gain, normalises) the heads of q and k, given as
    `qk_rows`; `rotary` from rotary(), `pos` int32 [batch * seq]."""
    _qk("slora_qk_rotary_fwd", [q.dt], batch, seq, head_dim, q, k, rotary, pos, eps, ctx_len, ws,
        stream)


def slora_qk_rotary_bwd(batch, seq, head_dim, q, k=None, rotary=None, pos=None, eps=RMS_EPS,
                        ctx_len=None, ws=None, stream=None):
    _qk("slora_qk_rotary_bwd", [q.dt, q.gdt], batch, seq, head_dim, q, k, rotary, pos, eps,
        ctx_len, ws, stream)


# ------------------------------------------- 8-bit activation checkpoints
ACT8_BLOCK = 32
BF = torch.bfloat16


def act8_empty(T, d, device="cuda"):
    """(codes, scales) of a checkpoint of [T x d] activations."""
    nb = (d + ACT8_BLOCK - 1) // ACT8_BLOCK
    return (torch.empty((T, nb * ACT8_BLOCK), dtype=torch.int8, device=device),
            torch.empty((T, nb), dtype=torch.uint8, device=device))


def act8(codes, scales, T, d) -> Act8:
    """The C struct of a checkpoint of [T x d] activations."""
    nb = (d + ACT8_BLOCK - 1) // ACT8_BLOCK
    if (codes.dtype is not torch.int8 or scales.dtype is not torch.uint8
            or codes.numel() != T * nb * ACT8_BLOCK or scales.numel() != T * nb
            or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError(f"a checkpoint of {T} x {d} activations is contiguous int8 "
                         f"[{T} x {nb * ACT8_BLOCK}] and uint8 [{T} x {nb}]")
    return Act8(codes.data_ptr() or None, scales.data_ptr() or None)


def _ref(c):
    return None if c is None else ctypes.byref(c)


def slora_act8_pack(X, codes, scales, stream=None):
    T, d = X.shape
    px, ldx = _rows(X, "X")
    c = act8(codes, scales, T, d)
    _here(X, codes, scales)
    _run_plain("slora_act8_pack", [dtype_code(X), T, d, px, ldx, ctypes.byref(c)], stream)


def slora_act8_unpack(codes, scales, X, stream=None):
    T, d = X.shape
    px, ldx = _rows(X, "X")
    c = act8(codes, scales, T, d)
    _here(X, codes, scales)
    _run_plain("slora_act8_unpack", [dtype_code(X), T, d, ctypes.byref(c), px, ldx], stream)


def slora_rmsnorm_fwd_act8(X, g, N, rstd=None, A=None, H=None, H8=None, N8=None, eps=RMS_EPS,
                           stream=None):
    """H8, N8: (codes, scales) of the checkpoints to write, or None."""
    T, d = X.shape
    h8 = None if H8 is None else act8(*H8, T, d)
    n8 = None if N8 is None else act8(*N8, T, d)
    args = [BF16, T, d, eps, _fit(X, "X", T * d, BF), _fit(A, "A", T * d, BF), _fit(g, "g", d, BF),
            _fit(H, "H", T * d, BF), _fit(N, "N", T * d, BF),
            _fit(rstd, "rstd", T, torch.float32), _ref(h8), _ref(n8)]
    _here(X, g, N, rstd, A, H, *(H8 or ()), *(N8 or ()))
    _run_plain("slora_rmsnorm_fwd_act8", args, stream)


def slora_rmsnorm_bwd_act8(H8, rstd, g, dN0, dX, dN1=None, dN2=None, dRes=None, stream=None):
    T, d = dN0.shape
    h8 = act8(*H8, T, d)
    args = [BF16, T, d, ctypes.byref(h8), _fit(rstd, "rstd", T, torch.float32), _fit(g, "g", d, BF),
            _fit(dN0, "dN0", T * d, BF), _fit(dN1, "dN1", T * d, BF), _fit(dN2, "dN2", T * d, BF),
            _fit(dRes, "dRes", T * d, BF), _fit(dX, "dX", T * d, BF)]
    _here(*H8, rstd, g, dN0, dN1, dN2, dRes, dX)
    _run_plain("slora_rmsnorm_bwd_act8", args, stream)


def slora_linear_bwd_act8(side, batch, seq, ctx_len, k, n, W, A, B, lora_scale, idx, X8_ctx,
                          XA_save, dY_ctx, dX_ctx, dA, dB, X8_out=None, dY_out=None, dX_out=None,
                          ws=None, stream=None):
    """slora_linear_bwd with the layer input given as checkpoints: X8_ctx and,
    for SLICE_IN_COLS, X8_out are (codes, scales)."""
    tok, keep, TC = _tokens(batch, seq, tuple(map(int, ctx_len)))
    n_idx = 0 if idx is None else idx.numel()
    T, r = batch * seq, A.shape[0]
    cols, rows = side == SLICE_IN_COLS, side == SLICE_OUT_ROWS
    xc = None if X8_ctx is None else act8(*X8_ctx, TC if cols else T, n_idx if cols else k)
    xo = None if X8_out is None else act8(*X8_out, T - TC, k)
    # an empty channel list is still a list: its address, never read, may be null
    pidx = _fit(idx, "idx", n_idx, torch.int32) or (None if idx is None else ptr(XA_save))
    f32 = torch.float32
    args = [dtype_code(W), ctypes.byref(tok), k, n, _fit(W, "W", n * k, BF), _fit(A, "A", r * k, BF),
            _fit(B, "B", n * r, BF), r, float(lora_scale), side, pidx, n_idx, _ref(xc), _ref(xo),
            _fit(XA_save, "XA_save", T * r, f32),
            _fit(dY_ctx, "dY_ctx", TC * n_idx if rows else T * n, BF),
            _fit(dY_out, "dY_out", (T - TC) * n, BF),
            _fit(dX_ctx, "dX_ctx", TC * n_idx if cols else T * k, BF),
            _fit(dX_out, "dX_out", (T - TC) * k, BF), _fit(dA, "dA", r * k, f32),
            _fit(dB, "dB", n * r, f32)]
    _here(W, A, B, idx, *(X8_ctx or ()), *(X8_out or ()), XA_save, dY_ctx, dY_out, dX_ctx, dX_out, dA, dB, ws)
    _run_scratch("slora_linear_bwd_act8", args, ws, stream)
    del keep
