"""Short convolution against its plain 64-bit form, every element.

Tolerance (layer_reference.check): half a step of the output's type plus a
number of fp32 roundings (2^-24) of the magnitudes summed.  Forward: the
window's sum has at most 2 W + 1 roundings, the activation's relative error
is that of exp2 (argument |u| log2 e: |u| + 2 roundings), a reciprocal and two
products; with |u| below 16 here that is under 64.  Gradients of the input
add as many again (128); those of the parameters one per token summed.
"""
import pytest
import torch

import gated_delta_rule_105_amd as kda
import layer_reference as ref
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(B, T, D, W, dtype, bias=True, state=True, lengths=None, fused=False, seed=0):
    g = torch.Generator().manual_seed(1000 + seed)
    dt = DT[dtype]
    cu = None
    if lengths is not None:
        B, T = 1, sum(lengths)
        cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32)
    S = B if cu is None else len(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = r(B, T, 2 * D + 3).to(dt)[..., 2: D + 2] if fused else r(B, T, D).to(dt)
    return dict(x=x, w=r(D, W) / 2, bias=r(D) if bias else None, init=r(S, W - 1, D).to(dt) if state else None,
                cu=cu, dy=r(B, T, D).to(dt), dfinal=r(S, W - 1, D).to(dt) if state else None)


def dev(t):
    # a slice stays a slice: copy what it was cut from
    if t is None:
        return None
    if t._base is not None and not t.is_contiguous():
        return t._base.cuda().as_strided(t.size(), t.stride(), t.storage_offset())
    return t.cuda()


CASES = {
    "one-token": dict(B=1, T=1, D=8, W=4, dtype="bf16"),
    "two-tokens-no-state": dict(B=1, T=2, D=3, W=4, dtype="f32", state=False),
    "one-channel": dict(B=2, T=9, D=1, W=2, dtype="bf16", bias=False),
    "odd-channels": dict(B=1, T=40, D=517, W=3, dtype="bf16"),
    "odd-channels-f32": dict(B=3, T=33, D=261, W=4, dtype="f32", bias=False),
    "rows-crossing-tiles": dict(B=5, T=13, D=64, W=4, dtype="bf16"),
    "long": dict(B=2, T=300, D=72, W=4, dtype="bf16", state=False),
    "long-f32": dict(B=1, T=519, D=130, W=2, dtype="f32"),
    "many-waves": dict(B=1, T=700, D=4096, W=4, dtype="bf16"),
    "packed": dict(B=1, T=0, D=40, W=4, dtype="bf16", lengths=[0, 1, 2, 3, 0, 0, 64, 17, 130, 1, 0]),
    "packed-f32": dict(B=1, T=0, D=19, W=3, dtype="f32", lengths=[70, 1, 0, 5, 2, 66], state=False),
    "packed-all-empty": dict(B=1, T=0, D=19, W=3, dtype="f32", lengths=[0, 0]),
    "slice": dict(B=2, T=37, D=50, W=4, dtype="bf16", fused=True),
    "slice-f32": dict(B=1, T=21, D=33, W=3, dtype="f32", fused=True),
}


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, act):
    p = inputs(**CASES[case])
    note(f"short_conv_forward {case} {act}")
    y, fin = kda.short_conv_forward(dev(p["x"]), dev(p["w"]), dev(p["bias"]), initial_state=dev(p["init"]),
                                    cu_seqlens=dev(p["cu"]), activation=act)
    torch.cuda.synchronize()
    ry, rf, my = ref.conv(p["x"], p["w"], p["bias"], p["init"], p["cu"], act)
    check("y", y, ry, my, 64)
    assert torch.equal(fin.cpu().double(), rf)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, act):
    p = inputs(**CASES[case], seed=1)
    note(f"short_conv_backward {case} {act}")
    g = kda.short_conv_backward(dev(p["x"]), dev(p["w"]), dev(p["dy"]), dev(p["bias"]), initial_state=dev(p["init"]),
                                dfinal=dev(p["dfinal"]), cu_seqlens=dev(p["cu"]), activation=act)
    torch.cuda.synchronize()
    rg, rm = ref.conv_grad(p["x"], p["w"], p["dy"], p["bias"], p["init"], p["dfinal"], p["cu"], act)
    n = p["x"].shape[0] * p["x"].shape[1]
    check("dx", g["dx"], rg["dx"], rm["dx"], 128)
    check("dweight", g["dweight"], rg["dweight"], rm["dweight"], 128 + n)
    for key, given, r in (("dbias", p["bias"], 128 + n), ("dinitial", p["init"], 128)):
        if given is None:
            assert g[key] is None
        else:
            check(key, g[key], rg[key], rm[key], r)


@pytest.mark.parametrize("N,D,W,dtype,fused", [(1, 8, 4, "bf16", False), (7, 5, 3, "bf16", True), (3, 129, 2, "f32", False),
                                               (64, 512, 4, "bf16", True), (2, 1, 4, "f32", True)])
def test_step_is_the_forward(N, D, W, dtype, fused):
    """Tokens one at a time against the whole sequences, bit for bit, and against the plain form."""
    T = 6
    p = inputs(B=N, T=T, D=D, W=W, dtype=dtype, fused=fused, seed=2)
    note(f"short_conv_step N={N} D={D} W={W} {dtype}")
    x, w, b = dev(p["x"]), dev(p["w"]), dev(p["bias"])
    y, fin = kda.short_conv_forward(x, w, b, initial_state=dev(p["init"]))
    state = dev(p["init"]).clone()
    for t in range(T):
        yt = kda.short_conv_step(x[:, t], w, state, b)
        torch.cuda.synchronize()
        assert torch.equal(yt, y[:, t])
    assert torch.equal(state, fin)
    ry, _, my = ref.conv(p["x"], p["w"], p["bias"], p["init"])
    check("y", y, ry, my, 64)


def test_resume():
    """A prompt in two calls, the first one's final state handed to the second, is the prompt in one."""
    p = inputs(B=2, T=90, D=48, W=4, dtype="bf16", seed=3)
    note("short_conv resume")
    x, w = dev(p["x"]), dev(p["w"])
    y, fin = kda.short_conv_forward(x, w, initial_state=dev(p["init"]))
    for cut in (1, 2, 41):
        ya, sa = kda.short_conv_forward(x[:, :cut].contiguous(), w, initial_state=dev(p["init"]))
        yb, sb = kda.short_conv_forward(x[:, cut:].contiguous(), w, initial_state=sa)
        assert torch.equal(torch.cat([ya, yb], 1), y) and torch.equal(sb, fin)


def test_nan_stays_in_its_windows():
    p = inputs(B=1, T=0, D=24, W=4, dtype="f32", lengths=[30, 50, 20], seed=4)
    note("short_conv nan")
    x, w, cu = dev(p["x"]), dev(p["w"]), dev(p["cu"])
    y, _ = kda.short_conv_forward(x, w, cu_seqlens=cu)
    dx = kda.short_conv_backward(x, w, dev(p["dy"]), cu_seqlens=cu)["dx"]
    x2 = x.clone()
    x2[0, 78, 5] = float("nan")
    y2, _ = kda.short_conv_forward(x2, w, cu_seqlens=cu)
    dx2 = kda.short_conv_backward(x2, w, dev(p["dy"]), cu_seqlens=cu)["dx"]
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 78:80, 5] = True  # the sequence ends at 80
    assert torch.equal(torch.isnan(y2), hit) and torch.equal(y2[~hit], y[~hit])
    hit[0, 75:80, 5] = True  # the tokens those windows read
    assert torch.equal(torch.isnan(dx2), hit) and torch.equal(dx2[~hit], dx[~hit])


def test_autograd_and_determinism():
    p = inputs(B=2, T=70, D=36, W=4, dtype="f32", seed=5)
    note("short_conv autograd")
    leaves = {k: dev(p[k]).requires_grad_() for k in ("x", "w", "bias", "init")}
    y, fin = kda.short_conv(leaves["x"], leaves["w"], leaves["bias"], initial_state=leaves["init"])
    ((y * dev(p["dy"])).sum() + (fin * dev(p["dfinal"])).sum()).backward()
    args = (dev(p["x"]), dev(p["w"]), dev(p["dy"]), dev(p["bias"]))
    g = kda.short_conv_backward(*args, initial_state=dev(p["init"]), dfinal=dev(p["dfinal"]))
    for k, name in (("x", "dx"), ("w", "dweight"), ("bias", "dbias"), ("init", "dinitial")):
        assert torch.equal(leaves[k].grad, g[name]), k
    # an output nobody used has no gradient: the same as zeros
    x = dev(p["x"]).requires_grad_()
    kda.short_conv(x, args[1])[0].sum().backward()
    assert torch.equal(x.grad, kda.short_conv_backward(args[0], args[1], torch.ones_like(args[2]))["dx"])
