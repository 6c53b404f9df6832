"""Workloads of the q/k rotation with per-head norms and of the 8-bit activation checkpoints.

Two groups of operators of a LoRA training layer, each in its plain form (elementary torch
operations in fp32) and as the calls of this package's library:

  q/k rotation   the rows of q and k, each head optionally RMS-normalised with a gain, rotated by
                 its position (half or interleaved pairs, all or the leading channels of a head,
                 one of four long-context scalings), forward and backward, on dense rows or on the
                 compact rows of the sliced projections (`slora_qk_rotary_fwd` / `_bwd`)
  checkpoints    activations kept for the backward pass as 8-bit integers with one power-of-two
                 scale per 32 channels: packing and unpacking (`slora_act8_pack` / `_unpack`), the
                 RMS norm that writes its checkpoints in the same pass and its backward from one
                 (`slora_rmsnorm_fwd_act8` / `_bwd_act8`), and the backward of a sliced LoRA linear
                 whose input is a checkpoint (`slora_linear_bwd_act8`)

`own` selects the library's calls in `run`; the plain form needs torch alone.
"""
import math

import torch

own = False

HALF, INTERLEAVED = "half", "interleaved"
BLOCK = 32  # channels that share a checkpoint's scale


# ------------------------------------------------------------------ cases
def listed():
    qk = {"kind": "qk", "dtype": "bf16", "grads": "f32", "layout": HALF, "dims": 128, "base": 10000.0,
          "scaling": "none", "factor": 1.0, "orig": 4096, "norm": False, "sliced": 0.0, "ctx": 1.0,
          "start": 0, "padded": False}
    lin = {"kind": "linear", "scale": 1.0}
    return [
        # one token far into a long context: a call whose cost is its latency
        {**qk, "name": "rotary fwd, one token", "step": "fwd", "batch": 1, "seq": 1, "heads": 32,
         "kv_heads": 8, "hd": 128, "scaling": "linear", "factor": 8.0, "start": 100_000,
         "layout": INTERLEAVED},
        # the Llama-3-8B-shaped layer at 8192 tokens a batch with a scaling by wavelength bands
        {**qk, "name": "rotary fwd, 16x512 grouped", "step": "fwd", "batch": 16, "seq": 512, "heads": 32,
         "kv_heads": 8, "hd": 128, "base": 500000.0, "scaling": "bands", "factor": 8.0, "orig": 8192},
        # rotation of a part of narrow heads, left-padded odd batch, gradients in fp32
        {**qk, "name": "rotary bwd, part of the head", "step": "bwd", "batch": 3, "seq": 1111, "heads": 12,
         "kv_heads": 4, "hd": 96, "dims": 48, "layout": INTERLEAVED, "scaling": "yarn", "factor": 4.0,
         "padded": True},
        # the Llama-2-7B-shaped attention projections with normalised heads
        {**qk, "name": "norm+rotary fwd, 4x1024", "step": "fwd", "batch": 4, "seq": 1024, "heads": 32,
         "kv_heads": 32, "hd": 128, "norm": True},
        # the training step's backward with gradients of the gains
        {**qk, "name": "norm+rotary bwd, 4x2048 grouped", "step": "bwd", "batch": 4, "seq": 2048,
         "heads": 32, "kv_heads": 8, "hd": 128, "norm": True, "base": 500000.0},
        # the sliced rows of the sparse q/k projections: half the channels on three quarters of the rows
        {**qk, "name": "norm+rotary sliced step", "step": "both", "batch": 4, "seq": 1024, "heads": 32,
         "kv_heads": 32, "hd": 128, "norm": True, "sliced": 0.5, "ctx": 0.75},
        # a checkpoint of the tiny FFN's intermediate rows, width no multiple of 128
        {"name": "checkpoint 77x688", "kind": "act8", "T": 77, "d": 688, "dtype": "bf16"},
        # the widest activation of the Llama-3-8B-shaped layer at 8192 tokens
        {"name": "checkpoint 8192x14336", "kind": "act8", "T": 8192, "d": 14336, "dtype": "bf16"},
        # residual add, norm and both of its checkpoints, then the norm's backward from one of them
        {"name": "norm with checkpoints 4096x4096", "kind": "norm", "T": 4096, "d": 4096},
        # the tiny layer's dense linear
        {**lin, "name": "linear bwd 1x256, 256->688", "side": "none", "batch": 1, "seq": 256, "ctx": 0.75,
         "k": 256, "n": 688, "r": 8, "keep": 1.0},
        # a sliced q projection, 4 x 1024 tokens, half the output channels of the context rows
        {**lin, "name": "linear bwd 4x1024, q sliced", "side": "out_rows", "batch": 4, "seq": 1024,
         "ctx": 0.75, "k": 4096, "n": 4096, "r": 16, "keep": 0.5},
        # a down projection that reads half its input channels on context rows
        {**lin, "name": "linear bwd 8x512, down sliced", "side": "in_cols", "batch": 8, "seq": 512,
         "ctx": 0.75, "k": 11008, "n": 4096, "r": 16, "keep": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["qk", "qk", "qk", "act8", "norm", "linear"])
    if kind == "qk":
        hd = rng.choice([64, 128, 128, 80, 96, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        tokens = _log(rng, 1, 200_000 // (heads + kv))
        batch = rng.choice([1, 1, 2, 5])
        batch = batch if batch <= tokens else 1
        norm = rng.random() < 0.6
        sliced = rng.choice([0.0, 0.0, 0.3, 0.5])
        scaling = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
        return {"kind": "qk", "dtype": rng.choice(["bf16", "bf16", "f32"]) if not sliced else "bf16",
                "grads": rng.choice(["bf16", "f32"]), "layout": rng.choice([HALF, INTERLEAVED]),
                "dims": rng.choice([hd, hd, hd // 2, hd // 4]), "base": rng.choice([10000.0, 500000.0]),
                "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                "orig": rng.choice([2048, 8192]), "norm": norm, "sliced": sliced,
                "ctx": 1.0 if not sliced else rng.choice([0.5, 0.75, 1.0]),
                "start": 0 if sliced else rng.choice([0, 0, 1000, 250_000]),
                "padded": rng.random() < 0.3 and not sliced, "step": rng.choice(["fwd", "bwd", "both"]),
                "batch": batch, "seq": max(1, tokens // batch), "heads": heads, "kv_heads": kv, "hd": hd}
    if kind == "act8":
        d = 8 * _log(rng, 8, 1792)
        return {"kind": "act8", "T": _log(rng, 1, min(16384, 100_000_000 // d)), "d": d,
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if kind == "norm":
        d = 8 * _log(rng, 8, 1024)
        return {"kind": "norm", "T": _log(rng, 1, min(16384, 16_000_000 // d)), "d": d}
    batch = rng.choice([1, 2, 4])
    return {"kind": "linear", "side": rng.choice(["none", "out_rows", "in_cols"]), "batch": batch,
            "seq": _log(rng, 4, 4096 // batch), "ctx": rng.choice([0.5, 0.75]), "k": 8 * _log(rng, 8, 700),
            "n": 8 * _log(rng, 8, 700), "r": rng.choice([4, 8, 16, 32]), "keep": rng.choice([0.3, 0.5, 0.7]),
            "scale": rng.choice([1.0, 2.0])}


# ------------------------------------------------------------- preparation
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _frequencies(c):
    """Angle per position of each rotated pair (radians) and the factor on the rotated channels."""
    half = c["dims"] // 2
    base, s = c["base"], c["factor"]
    if c["scaling"] == "ntk":
        base = base * s ** (c["dims"] / (c["dims"] - 2))
    f = [base ** (-2.0 * i / c["dims"]) for i in range(half)]
    if c["scaling"] == "linear":
        return [v / s for v in f], 1.0
    if c["scaling"] == "bands":  # below 1 and above 4 turns over the original context
        turns = [c["orig"] * v / (2.0 * math.pi) for v in f]
        mix = [min(1.0, max(0.0, (t - 1.0) / (4.0 - 1.0))) for t in turns]
        return [m * v + (1.0 - m) * v / s for m, v in zip(mix, f)], 1.0
    if c["scaling"] == "yarn":  # a ramp over the pairs between 32 and 1 turns
        def pair(turns):
            return c["dims"] * math.log(c["orig"] / (2.0 * math.pi * turns)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), c["dims"] - 1)
        mix = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(half)]
        return [m * v / s + (1.0 - m) * v for m, v in zip(mix, f)], 0.1 * math.log(s) + 1.0
    return f, 1.0


def _context_lengths(c):
    """Context rows of each sequence: `ctx` of it, one row fewer in every second sequence."""
    return [max(0, int(c["ctx"] * c["seq"]) - (b % 2 if c["ctx"] < 1.0 else 0)) for b in range(c["batch"])]


def _randn(shape, gen, dt=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda").to(dt)


def _activations(T, d, gen, dt=torch.bfloat16):
    """Rows as a trained network has them: a few channels far larger than the rest."""
    loud = 1.0 + 15.0 * (torch.rand(d, generator=gen, device="cuda") < 0.01)
    return (torch.randn((T, d), generator=gen, device="cuda") * loud).to(dt)


def _power(e):
    """2^e in fp32 for whole -126 <= e <= 127, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _pack_plain(X):
    """Codes and scale bytes: each 32 channels of a row share 2^(e - 6), e = floor(log2(largest))."""
    T, d = X.shape
    x = torch.nn.functional.pad(X.float(), (0, -d % BLOCK)).view(T, -1, BLOCK)
    e = torch.frexp(x.abs().amax(2)).exponent.int() - 1
    e = e.clamp(min=-120)
    codes = torch.round(x * _power(6 - e)[:, :, None]).clamp(-127, 127)
    return codes.to(torch.int8).reshape(T, -1), (e + 127).to(torch.uint8)


def _values(codes, scales, d):
    """The fp32 values that a checkpoint's codes and scale bytes stand for."""
    return (codes.view(*scales.shape, BLOCK).float() * _power(scales.int() - 133)[:, :, None]).reshape(codes.shape)[:, :d]


def _split_rows(c):
    """Full-layout indices of the context and of the output rows."""
    lens = torch.tensor(_context_lengths(c))
    is_ctx = (torch.arange(c["seq"])[None] < lens[:, None]).reshape(-1)
    return torch.nonzero(is_ctx)[:, 0].cuda(), torch.nonzero(~is_ctx)[:, 0].cuda()


def _prepare_qk(c, gen):
    T = c["batch"] * c["seq"]
    dt, gdt = _dtype(c["dtype"]), _dtype(c["grads"]) if c["dtype"] == "bf16" else torch.float32
    freq, mscale = _frequencies(c)
    # a left-padded batch keeps position 0 on its padding
    pos = torch.arange(c["seq"], dtype=torch.int32)[None].repeat(c["batch"], 1) + c["start"]
    if c["padded"]:
        for b in range(c["batch"]):
            pos[b] = (pos[b] - (b * 37) % c["seq"]).clamp(min=0)
    plain_pos = c["start"] == 0 and not c["padded"]
    st = {"case": c, "pos": pos.reshape(-1).cuda(), "given_pos": not plain_pos, "mscale": mscale,
          "freq": torch.tensor(freq, dtype=torch.float64).cuda(), "parts": []}
    if c["sliced"]:
        st["ctx_rows"], st["out_rows"] = _split_rows(c)
    kh = c["hd"] - int(c["sliced"] * c["hd"])
    sets = torch.rand((c["kv_heads"], c["hd"]), generator=gen, device="cuda")
    kept = torch.sort(torch.topk(sets, kh, 1).indices, 1).values
    for heads in (c["heads"], c["kv_heads"]):
        n = heads * c["hd"]
        p = {"heads": heads, "g": None, "dg": None}
        if c["norm"]:
            p["g"] = (1.0 + 0.1 * torch.randn(c["hd"], generator=gen, device="cuda")).to(dt)
        if c["sliced"]:
            group = torch.arange(heads, device="cuda") // (heads // c["kv_heads"])
            idx = (kept[group] + c["hd"] * torch.arange(heads, device="cuda")[:, None]).reshape(-1)
            p["idx"] = idx.int()
            p["X_ctx"] = _randn((len(st["ctx_rows"]), len(idx)), gen, dt)
            p["X_out"] = _randn((len(st["out_rows"]), n), gen, dt)
        else:
            p["X"] = _activations(T, n, gen, dt)
        if c["step"] != "bwd":
            p["Y"] = torch.empty((T, n), dtype=dt, device="cuda")
        if c["step"] != "fwd":
            p["dY"] = _randn((T, n), gen, gdt)
            if c["sliced"]:
                p["dX_ctx"], p["dX_out"] = torch.empty_like(p["X_ctx"]), torch.empty_like(p["X_out"])
            else:
                p["dX"] = torch.empty_like(p["X"])
            if c["norm"]:
                p["dg"] = torch.empty(c["hd"], device="cuda")
        st["parts"].append(p)
    return st


def _prepare_norm(c, gen):
    T, d = c["T"], c["d"]
    return {"case": c, "X": _activations(T, d, gen), "A": _randn((T, d), gen),
            "g": (1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")).bfloat16(),
            "dN": _randn((T, d), gen), "dRes": _randn((T, d), gen),
            **{k: torch.empty((T, d), dtype=torch.bfloat16, device="cuda") for k in ("H", "N", "dX", "N8v")},
            "rstd": torch.empty(T, device="cuda"),
            **{k: (torch.empty((T, d + -d % BLOCK), dtype=torch.int8, device="cuda"),
                   torch.empty((T, (d + BLOCK - 1) // BLOCK), dtype=torch.uint8, device="cuda"))
               for k in ("H8", "N8")}}


def _prepare_linear(c, gen):
    T, k, n, r = c["batch"] * c["seq"], c["k"], c["n"], c["r"]
    rows_c, rows_o = _split_rows(c)
    st = {"case": c, "ctx_rows": rows_c, "out_rows": rows_o, "idx": None}
    sliced = {"none": 0, "out_rows": n, "in_cols": k}[c["side"]]
    if sliced:
        keep = max(1, int(c["keep"] * sliced))
        pick = torch.topk(torch.rand(sliced, generator=gen, device="cuda"), keep).indices
        st["idx"] = torch.sort(pick).values.int()
    ni = 0 if st["idx"] is None else len(st["idx"])
    W = torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5
    # rows of W are the sliced channels: the transposed copy for sliced inputs
    st["W"] = (W.t() if c["side"] == "in_cols" else W).contiguous().bfloat16()
    st["A"] = (torch.randn((r, k), generator=gen, device="cuda") * k ** -0.5).bfloat16()
    st["B"] = (torch.randn((n, r), generator=gen, device="cuda") * 0.05).bfloat16()
    grad = 1e-3
    if c["side"] == "in_cols":
        xs = [_activations(len(rows_c), ni, gen), _activations(len(rows_o), k, gen)]
        st["dY_ctx"], st["dY_out"] = (_randn((T, n), gen, torch.float32) * grad).bfloat16(), None
    else:
        xs = [_activations(T, k, gen), None]
        nc = n if c["side"] == "none" else ni
        rc, ro = (T, 0) if c["side"] == "none" else (len(rows_c), len(rows_o))
        st["dY_ctx"] = (_randn((rc, nc), gen, torch.float32) * grad).bfloat16()
        st["dY_out"] = (_randn((ro, n), gen, torch.float32) * grad).bfloat16() if ro else None
    st["X8"] = [None if x is None else _pack_plain(x) for x in xs]
    xa = [None if x is None else x.float() for x in xs]
    A = st["A"].float()
    if c["side"] == "in_cols":
        XA = torch.empty((T, r), device="cuda")
        XA[rows_c] = xa[0] @ A[:, st["idx"].long()].t()
        XA[rows_o] = xa[1] @ A.t()
    else:
        XA = xa[0] @ A.t()
    st["XA"] = XA
    st["dX"] = [None if x is None else torch.empty_like(x) for x in xs]
    st["dA"], st["dB"] = torch.empty((r, k), device="cuda"), torch.empty((n, r), device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["kind"] == "qk":
        return _prepare_qk(case, gen)
    if case["kind"] == "act8":
        X = _activations(case["T"], case["d"], gen, _dtype(case["dtype"]))
        return {"case": case, "X": X, "back": torch.empty_like(X),
                "codes": torch.empty((case["T"], case["d"] + -case["d"] % BLOCK), dtype=torch.int8, device="cuda"),
                "scales": torch.empty((case["T"], (case["d"] + BLOCK - 1) // BLOCK), dtype=torch.uint8,
                                      device="cuda")}
    if case["kind"] == "norm":
        return _prepare_norm(case, gen)
    return _prepare_linear(case, gen)


# ---------------------------------------------------------- the plain form
EPS = 1e-5


def _full_rows(st, p, n):
    """Sliced rows at full width: a context row's skipped channels are zero."""
    x = torch.zeros((len(st["ctx_rows"]) + len(st["out_rows"]), n), device="cuda")
    x[st["ctx_rows"][:, None], p["idx"].long()[None]] = p["X_ctx"].float()
    x[st["out_rows"]] = p["X_out"].float()
    return x


def _turn(y, cos, sin, c):
    """Rotates the leading `dims` channels of heads y [T, heads, hd] by the pairs' angles."""
    dims, out = c["dims"], y.clone()
    if c["layout"] == HALF:
        a, b = y[..., :dims // 2], y[..., dims // 2:dims]
        out[..., :dims // 2] = a * cos - b * sin
        out[..., dims // 2:dims] = b * cos + a * sin
    else:
        a, b = y[..., 0:dims:2], y[..., 1:dims:2]
        out[..., 0:dims:2] = a * cos - b * sin
        out[..., 1:dims:2] = b * cos + a * sin
    return out


def _plain_qk(st):
    c = st["case"]
    hd, outs = c["hd"], []
    angle = st["pos"].double()[:, None] * st["freq"][None]
    cos = (angle.cos() * st["mscale"]).float()[:, None]
    sin = (angle.sin() * st["mscale"]).float()[:, None]
    for p in st["parts"]:
        n = p["heads"] * hd
        x = (_full_rows(st, p, n) if c["sliced"] else p["X"].float()).view(-1, p["heads"], hd)
        if c["norm"]:
            rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            g = p["g"].float()
        if c["step"] != "bwd":
            y = _turn(x * rstd * g if c["norm"] else x, cos, sin, c)
            outs.append(y.reshape(-1, n).to(_dtype(c["dtype"])))
        if c["step"] != "fwd":
            dn = _turn(p["dY"].float().view(-1, p["heads"], hd), cos, -sin, c)
            if c["norm"]:
                outs.append((dn * x * rstd).sum((0, 1)))
                u = dn * g
                dn = rstd * u - x * rstd ** 3 * (u * x).mean(-1, keepdim=True)
            dx = dn.reshape(-1, n).to(_dtype(c["dtype"]))
            if c["sliced"]:
                outs += [dx[st["ctx_rows"][:, None], p["idx"].long()[None]], dx[st["out_rows"]]]
            else:
                outs.append(dx)
    return outs


def _plain_norm(st):
    d = st["case"]["d"]
    h = (st["X"].float() + st["A"].float()).bfloat16()
    x, g = h.float(), st["g"].float()
    rstd = torch.rsqrt((x * x).mean(1) + EPS)
    N = (x * rstd[:, None] * g).bfloat16()
    back = _values(*_pack_plain(h), d)  # the backward reads the residual sum's checkpoint
    u = st["dN"].float() * g
    dX = st["dRes"].float() + rstd[:, None] * u - back * rstd[:, None] ** 3 * (u * back).mean(1, keepdim=True)
    return [N, rstd, _values(*_pack_plain(N), d).bfloat16(), dX.bfloat16()]


def _plain_linear(st):
    c = st["case"]
    k, s, A, B, W = c["k"], c["scale"], st["A"].float(), st["B"].float(), st["W"].float()
    XA, rc, ro = st["XA"], st["ctx_rows"], st["out_rows"]
    ix = None if st["idx"] is None else st["idx"].long()
    if c["side"] == "none":
        x, dy = _values(*st["X8"][0], k), st["dY_ctx"].float()
        p = dy @ B
        return [(dy @ W + s * (p @ A)).bfloat16(), s * (p.t() @ x), s * (dy.t() @ XA)]
    if c["side"] == "out_rows":
        x, dyc = _values(*st["X8"][0], k), st["dY_ctx"].float()
        dyo = torch.zeros((0, c["n"]), device="cuda") if st["dY_out"] is None else st["dY_out"].float()
        dX, p = torch.empty((len(x), k), device="cuda"), torch.empty((len(x), c["r"]), device="cuda")
        p[rc], p[ro] = dyc @ B[ix], dyo @ B
        dX[rc], dX[ro] = dyc @ W[ix] + s * (p[rc] @ A), dyo @ W + s * (p[ro] @ A)
        dB = s * (dyo.t() @ XA[ro])
        dB[ix] += s * (dyc.t() @ XA[rc])
        return [dX.bfloat16(), s * (p.t() @ x), dB]
    xc, xo = _values(*st["X8"][0], len(ix)), _values(*st["X8"][1], k)
    dy = st["dY_ctx"].float()
    p = dy @ B
    dXc = dy[rc] @ W[ix].t() + s * (p[rc] @ A[:, ix])
    dXo = dy[ro] @ W.t() + s * (p[ro] @ A)
    dA = s * (p[ro].t() @ xo)
    dA[:, ix] += s * (p[rc].t() @ xc)
    return [dXc.bfloat16(), dXo.bfloat16(), dA, s * (dy.t() @ XA)]


# ---------------------------------------------------- the library's calls
def _own_qk(st):
    from contextual_sparsity_lora_svd_b200 import _lib as L
    c = st["case"]
    rot = L.rotary(layout=c["layout"], dims=c["dims"], base=c["base"], scaling=c["scaling"],
                   factor=c["factor"], orig_len=c["orig"])
    q, k = (L.qk_rows(**{a: v for a, v in p.items()}) for p in st["parts"])
    args = (c["batch"], c["seq"], c["hd"], q, k)
    kw = {"rotary": rot, "pos": st["pos"] if st["given_pos"] else None, "eps": EPS,
          "ctx_len": _context_lengths(c) if c["sliced"] else None}
    if c["step"] != "bwd":
        L.slora_qk_rotary_fwd(*args, **kw)
    if c["step"] != "fwd":
        L.slora_qk_rotary_bwd(*args, **kw)
    outs = []
    for p in st["parts"]:
        outs += [p[a] for a in ("Y", "dg", "dX", "dX_ctx", "dX_out") if p.get(a) is not None]
    return outs


def _own(st):
    from contextual_sparsity_lora_svd_b200 import _lib as L
    c = st["case"]
    if c["kind"] == "qk":
        return _own_qk(st)
    if c["kind"] == "act8":
        L.slora_act8_pack(st["X"], st["codes"], st["scales"])
        L.slora_act8_unpack(st["codes"], st["scales"], st["back"])
        return [st["back"]]
    if c["kind"] == "norm":
        L.slora_rmsnorm_fwd_act8(st["X"], st["g"], st["N"], st["rstd"], A=st["A"], H=st["H"], H8=st["H8"],
                                 N8=st["N8"], eps=EPS)
        L.slora_act8_unpack(*st["N8"], st["N8v"])
        L.slora_rmsnorm_bwd_act8(st["H8"], st["rstd"], st["g"], st["dN"], st["dX"], dRes=st["dRes"])
        return [st["N"], st["rstd"], st["N8v"], st["dX"]]
    side = {"none": L.SLICE_NONE, "out_rows": L.SLICE_OUT_ROWS, "in_cols": L.SLICE_IN_COLS}[c["side"]]
    L.slora_linear_bwd_act8(side, c["batch"], c["seq"], _context_lengths(c), c["k"], c["n"], st["W"], st["A"],
                            st["B"], c["scale"], st["idx"], st["X8"][0], st["XA"], st["dY_ctx"], st["dX"][0],
                            st["dA"], st["dB"], X8_out=st["X8"][1], dY_out=st["dY_out"], dX_out=st["dX"][1])
    return [x for x in st["dX"] if x is not None] + [st["dA"], st["dB"]]


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "qk":
        return _plain_qk(state)
    if kind == "act8":
        d, dt = state["case"]["d"], state["X"].dtype
        return [_values(*_pack_plain(state["X"]), d).to(dt)]
    return _plain_norm(state) if kind == "norm" else _plain_linear(state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["kind"] == "qk":
        es = 4 if c["dtype"] == "f32" else 2
        gs = 2 if es == 2 and c["grads"] == "bf16" else 4
        lens = _context_lengths(c)
        T, tc, n = c["batch"] * c["seq"], sum(lens), (c["heads"] + c["kv_heads"]) * c["hd"]
        kh = (c["hd"] - int(c["sliced"] * c["hd"])) / c["hd"]
        x = es * n * (tc * kh + (T - tc) if c["sliced"] else T)  # the rows of q and k as they are held
        passes = {"fwd": x + es * T * n, "bwd": x + gs * T * n + x}
        passes["both"] = x + es * T * n + gs * T * n + x
        norm = 4 if c["norm"] else 0
        return {"bytes": passes[c["step"]],
                "flops": T * n * (3 + norm) * {"fwd": 1, "bwd": 2 if norm else 1, "both": 3 if norm else 2}[c["step"]]}
    if c["kind"] == "act8":
        es, n = 4 if c["dtype"] == "f32" else 2, c["T"] * c["d"]
        return {"bytes": n * (2 * es + 1) + n // BLOCK, "flops": 4 * n}
    if c["kind"] == "norm":
        n = c["T"] * c["d"]
        # X, A, dN and dRes read; N, its checkpoint's values and dX written
        return {"bytes": n * 2 * 7 + 4 * c["T"], "flops": 20 * n}
    T, k, n, r = c["batch"] * c["seq"], c["k"], c["n"], c["r"]
    tc = sum(_context_lengths(c))
    to = T - tc
    if c["side"] == "none":
        x, dy, w = T * k, T * n, 2.0 * T * n * k
    elif c["side"] == "out_rows":
        ni = max(1, int(c["keep"] * n))
        x, dy, w = T * k, tc * ni + to * n, 2.0 * k * (tc * ni + to * n)
    else:
        ni = max(1, int(c["keep"] * k))
        x, dy, w = tc * ni + to * k, T * n, 2.0 * n * (tc * ni + to * k)
    return {"bytes": x + x / BLOCK + 2 * dy + 2 * n * k + 2 * x + 2 * r * (n + k) + 4 * T * r + 4 * r * (n + k),
            "flops": w + 4.0 * r * (x + dy)}


# ------------------------------------------------------------ in 64 bits
def _exact_qk(st):
    c = st["case"]
    hd, dims, outs = c["hd"], c["dims"], []
    freq, m = _frequencies(c)
    T = c["batch"] * c["seq"]
    angle = torch.outer(st["pos"].double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    unit = torch.polar(torch.full_like(angle, m), angle)[:, None]  # a pair is a complex number

    def rotate(y, w):
        z = y[..., :dims].reshape(T, -1, 2, dims // 2).transpose(2, 3) if c["layout"] == HALF else \
            y[..., :dims].reshape(T, -1, dims // 2, 2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * w)
        z = z.transpose(2, 3) if c["layout"] == HALF else z
        return torch.cat([z.reshape(T, -1, dims), y[..., dims:]], -1)

    for p in st["parts"]:
        if c["sliced"]:
            x = torch.zeros((T, p["heads"] * hd), dtype=torch.float64, device="cuda")
            rows = torch.zeros_like(x[st["ctx_rows"]])
            rows[:, p["idx"].long()] = p["X_ctx"].double()
            x[st["ctx_rows"]], x[st["out_rows"]] = rows, p["X_out"].double()
        else:
            x = p["X"].double()
        x = x.view(T, p["heads"], hd)
        inv = ((x.square().sum(-1) / hd + EPS) ** -0.5)[..., None] if c["norm"] else torch.ones((), device="cuda")
        g = p["g"].double() if c["norm"] else torch.ones((), dtype=torch.float64, device="cuda")
        xhat = x * inv
        if c["step"] != "bwd":
            outs.append(rotate(xhat * g, unit).reshape(T, -1))
        if c["step"] != "fwd":
            dn = rotate(p["dY"].double().view(T, p["heads"], hd), unit.conj())
            dx = dn
            if c["norm"]:
                outs.append(torch.einsum("thc,thc->c", dn, xhat))
                dx = inv * (dn * g - xhat * ((dn * g * xhat).sum(-1, keepdim=True) / hd))
            dx = dx.reshape(T, -1)
            if c["sliced"]:
                outs += [dx[st["ctx_rows"]][:, p["idx"].long()], dx[st["out_rows"]]]
            else:
                outs.append(dx)
    return outs


def _step64(exponent):
    """The power of two whose biased 64-bit exponent this is."""
    return (exponent << 52).view(torch.float64)


def _exact_values(X):
    """Values of the checkpoint of X: each block's step is 2^-6 of the largest power of two in it."""
    T, d = X.shape
    x = torch.cat([X.double(), torch.zeros((T, -d % BLOCK), dtype=torch.float64, device="cuda")], 1)
    x = x.view(T, -1, BLOCK)
    top = x.abs().max(2, keepdim=True).values
    step = _step64((top.view(torch.int64) >> 52).clamp(min=1023 - 120) - 6)  # the exponent's own bits
    return ((x / step).round().clamp(-127, 127) * step).reshape(T, -1)[:, :d]


def _held(codes, scales, d):
    step = _step64(scales.long() + 1023 - 133).repeat_interleave(BLOCK, 1)
    return (codes.double() * step)[:, :d]


def _exact_linear(st):
    c = st["case"]
    s, W, A, B, XA = c["scale"], st["W"].double(), st["A"].double(), st["B"].double(), st["XA"].double()
    T, k, n = c["batch"] * c["seq"], c["k"], c["n"]
    rc, ro = st["ctx_rows"], st["out_rows"]
    # the same linear over full-width rows whose skipped channels are zero
    if c["side"] == "in_cols":
        W, ix = W.t(), st["idx"].long()
        x = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        x[rc[:, None], ix[None]] = _held(*st["X8"][0], len(ix))
        x[ro] = _held(*st["X8"][1], k)
        dy = st["dY_ctx"].double()
    else:
        x = _held(*st["X8"][0], k)
        dy = torch.zeros((T, n), dtype=torch.float64, device="cuda")
        if c["side"] == "none":
            dy[:] = st["dY_ctx"].double()
        else:
            dy[rc[:, None], st["idx"].long()[None]] = st["dY_ctx"].double()
            if st["dY_out"] is not None:
                dy[ro] = st["dY_out"].double()
    dX = dy @ (W + s * (B @ A))
    dA, dB = s * ((dy @ B).t() @ x), s * (dy.t() @ XA)
    if c["side"] == "in_cols":
        return [dX[rc][:, ix], dX[ro], dA, dB]
    return [dX, dA, dB]


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "qk":
        return _exact_qk(st)
    if case["kind"] == "act8":
        return [_exact_values(st["X"])]
    if case["kind"] == "linear":
        return _exact_linear(st)
    h = (st["X"].double() + st["A"].double()).bfloat16()  # the norm reads the rounded residual sum
    x, g = h.double(), st["g"].double()
    inv = (x.square().sum(1, keepdim=True) / case["d"] + EPS) ** -0.5
    held, u = _exact_values(h), st["dN"].double() * g
    dX = st["dRes"].double() + inv * u - held * inv ** 3 * ((u * held).sum(1, keepdim=True) / case["d"])
    return [x * inv * g, inv[:, 0], None, dX]
