"""layers.DecoderStack with its options: head norms and other rotations of q and
k (slora_qk_rotary_*), and 8-bit checkpoints of what the backward reads
(slora_rmsnorm_*_act8, slora_linear_bwd_act8), each alone and together, against
a float64 autograd step on the channel sets that the run chose."""
import numpy as np
import pytest
import torch

from contextual_sparsity_lora_svd_b200 import _lib as L
from tests import qk_reference as ref
from tests.helpers import assert_close, dev, host, rel_frob
from tests.test_gpu_stack import _rb, make_stack

pytestmark = pytest.mark.gpu

# A checkpoint's step is at most 2 max / 127 of its block of 32 values, and its rounding error at
# most half a step, evenly spread: rms step / sqrt(12) <= max / 220.  The largest of 32 normal values
# is 2.1 sigma, so a checkpoint of normal values is off by at most 2.1 / 220 = 1e-2 of its norm
# (independent of what it multiplies, so a sum over tokens is off by the same part of its norm).
CKPT = 1e-2
# What bf16 storage alone does to the step is computed: the float64 step with every stored tensor
# and its gradient rounded to bf16.  Over these cases it takes the output 5.9e-3 to 6.8e-3, the input
# gradient 7.2e-3 to 1.04e-2 and a LoRA gradient up to 1.7e-2 from the exact step (head norms and a
# longer rotation's factor sharpen the softmax, so the fixed bounds of the plain step, 1e-2 and 2e-2,
# lie below or at the roundings themselves).  The kernels round at a few more places that it does not
# model (the gate's and up's gradients, the softmax's terms before their division): at most as
# many again, independent, so sqrt(2) of it, here 1.5.
ROUNDINGS = 1.5

OPTIONS = [
    dict(qk_norm=True),
    dict(rotary=dict(layout="interleaved", dims=32, base=500000.0)),
    dict(act8=True),
    dict(act8=True, qk_norm=True, rotary=dict(scaling="yarn", factor=4.0, orig_len=32)),
    dict(act8=True, qk_norm=True, rotary=dict(layout="interleaved", dims=24, scaling="bands", factor=8.0,
                                              orig_len=64)),
]


def _case(seed, H, KV, hd, nl=3, b=2, seq=96):
    lays, devs = make_stack(nl, 256, H, KV, hd, 688, 8, 8, seed=seed)
    rng = np.random.default_rng(seed + 1)
    for lay, w in zip(lays, devs):
        for g in ("gq", "gk"):
            lay[g] = _rb(1.0 + 0.1 * rng.normal(size=hd))
            w[g] = dev(lay[g], torch.bfloat16)
    X, dY = _rb(rng.normal(size=(b * seq, 256))), _rb(rng.normal(size=(b * seq, 256)))
    return lays, devs, X, dY


def _run(devs, H, KV, hd, b, seq, ctx, qk_s, ffn_s, X, dY, **options):
    from contextual_sparsity_lora_svd_b200.layers import DecoderStack
    if options.get("rotary"):
        options["rotary"] = L.rotary(**options["rotary"])
    run = DecoderStack(devs, 256, H, KV, hd, 688, 8, 8, 1.0, b, seq, ctx, qk_s, ffn_s,
                       dev(X, torch.bfloat16), dev(dY, torch.bfloat16), **options)
    ws = torch.empty(run.workspace_bytes(), dtype=torch.uint8, device="cuda")
    run.step(ws)
    torch.cuda.synchronize()
    return run, ws


@pytest.mark.parametrize("H,KV,hd", [(4, 4, 64), (4, 2, 128)])
@pytest.mark.parametrize("options", OPTIONS, ids=lambda o: "+".join(o))
def test_step_with_options_matches_float64(H, KV, hd, options):
    nl, b, seq, ctx = 3, 2, 96, [96, 61]
    qk_s, ffn_s = [0.0, 0.5, 0.25], [0.0, 0.5, 0.7]
    lays, devs, X, dY = _case(31 + hd, H, KV, hd)
    run, _ = _run(devs, H, KV, hd, b, seq, ctx, qk_s, ffn_s, X, dY, **options)
    sets = []
    for l in range(nl):
        kh, kf = run.kh[l], run.k_ffn[l]
        qk = None if run.idx_qk[l] is None else host(run.idx_qk[l]).astype(np.int64)
        sets.append((None if qk is None else qk[:H * kh],
                     None if qk is None else qk[H * kh:(H + KV) * kh],
                     host(run.idx_ffn[l])[:kf].astype(np.int64)))
    if not options.get("qk_norm"):
        lays = [{k: v for k, v in lay.items() if k not in ("gq", "gk")} for lay in lays]
    turn = dict(options.get("rotary", {}))
    layout, dims = turn.pop("layout", "half"), turn.pop("dims", 0) or hd
    freq, m = ref.frequencies(dims, **turn)
    keep = ("W", "A", "B", "g")
    args = (X, dY, [{k: v for k, v in lay.items() if k[0] in keep or k == "scale"} for lay in lays],
            b, seq, ctx, H, KV, hd, sets, np.tile(np.arange(seq), b), freq, m, dims, layout)
    y, dX, grads = ref.stack(*args)
    ry, rdX, rgrads = ref.stack(*args, stored=True)
    more = CKPT if options.get("act8") else 0.0
    assert_close(host(run.y), y, ROUNDINGS * rel_frob(ry, y), "output")
    assert_close(host(run.dX), dX, ROUNDINGS * rel_frob(rdX, dX) + more, "input gradient")
    for l in range(nl):
        for key, val in grads[l].items():
            assert_close(host(run.grads[l][key]), val,
                         ROUNDINGS * rel_frob(rgrads[l][key], val) + more, f"layer {l} {key}")


def test_checkpoints_leave_the_forward_as_it_was():
    H, KV, hd, ctx = 4, 2, 64, [80, 96]
    qk_s, ffn_s = [0.5, 0.0, 0.5], [0.5, 0.5, 0.0]
    _, devs, X, dY = _case(5, H, KV, hd)
    plain, _ = _run(devs, H, KV, hd, 2, 96, ctx, qk_s, ffn_s, X, dY)
    small, _ = _run(devs, H, KV, hd, 2, 96, ctx, qk_s, ffn_s, X, dY, act8=True)
    assert torch.equal(plain.y, small.y)
    for l in range(3):
        assert torch.equal(plain.saved[l]["Qr"], small.saved[l]["Qr"])
        assert torch.equal(plain.saved[l]["O"], small.saved[l]["O"])
        assert small.saved[l]["n1"].data_ptr() == small.saved[0]["n1"].data_ptr()
    # the linears that read no checkpoint and whose dY passed through none
    assert torch.equal(plain.grads[2]["dBd"], small.grads[2]["dBd"])
    assert torch.equal(plain.grads[2]["dAg"], small.grads[2]["dAg"])


def test_the_default_rotation_by_either_call():
    """rotary=L.rotary() states the default rotation; the other call's angles are more exact, and
    its packed q and k differ from the default's by one rounding of bf16 at most plus 1e-5."""
    H, KV, hd, ctx = 4, 2, 64, [80, 96]
    _, devs, X, dY = _case(8, H, KV, hd, nl=1)
    a, _ = _run(devs, H, KV, hd, 2, 96, ctx, [0.5], [0.5], X, dY)
    b, _ = _run(devs, H, KV, hd, 2, 96, ctx, [0.5], [0.5], X, dY, rotary={})
    for key in ("Qr", "Kr"):
        p, q = a.saved[0][key].double(), b.saved[0][key].double()
        pair = p.view(-1, 2, hd // 2).norm(dim=1, keepdim=True).expand(-1, 2, -1).reshape(p.shape)
        assert ((p - q).abs() <= (2 ** -7 + 1e-5) * pair).all()


def test_options_replay_from_two_graphs_that_share_a_workspace():
    H, KV, hd, ctx = 4, 2, 64, [80, 33]
    _, devs, X, dY = _case(13, H, KV, hd, nl=2)
    options = dict(act8=True, qk_norm=True, rotary=dict(scaling="linear", factor=2.0))
    run, ws = _run(devs, H, KV, hd, 2, 96, ctx, [0.5, 0.0], [0.5, 0.5], X, dY, **options)
    other, ws2 = _run(devs, H, KV, hd, 2, 96, ctx, [0.0, 0.5], [0.5, 0.0], X, dY, **options)
    if ws2.numel() > ws.numel():
        ws = ws2
    want = [(r.y.clone(), r.gflat.clone()) for r in (run, other)]
    s, graphs = torch.cuda.Stream(), []
    for r in (run, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r.step(ws, s)
        graphs.append(g)
    for _ in range(2):
        for r, g, (y, grads) in zip((run, other), graphs, want):
            r.y.zero_()
            r.gflat.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(r.y, y)
            # dQ's atomic order moves its last bits (some 2^-22 of its terms): of the values rounded
            # to bf16 after it one in 2^13 lands a step of 2^-8 further, 2^-6.5 * 2^-8 = 4e-5 of
            # the norm for each rounding on the way, and there are fewer than seven
            assert_close(host(r.gflat), host(grads), 3e-4, "replayed gradients")
