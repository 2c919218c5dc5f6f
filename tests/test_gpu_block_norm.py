"""The norms at a block's end against their plain 64-bit forms, every element.

Tolerance (layer_reference.check): half a step of the output's type plus fp32
roundings (2^-24) of the magnitudes.  The statistic adds up to 8192 squares, a
lane 32 of them and 256 lanes in a tree: under 64, and its root and division
4; a gate's exponential is off by |z| + 3, which the magnitudes carry, and a
product has some 10 factors: under 128 together.  The parameters' gradients
add one term a row.
"""
import pytest
import torch

import block_reference as ref
import gated_delta_rule_105_amd as kda
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
N = 128


def cut(gen, rows, width, dt, fused):
    """[*rows, width], a slice that starts at an odd element of a wider tensor with `fused`."""
    if not fused:
        return torch.randn(*rows, width, generator=gen).to(dt).cuda()
    return torch.randn(*rows, width + 5, generator=gen).to(dt).cuda()[..., 3: 3 + width]


# every way a row is spread: single channels or vectors, lanes and loads a row
GATED = {
    "one": dict(rows=(1,), H=1, d=1, dtype="f32"),
    "odd": dict(rows=(5,), H=3, d=13, dtype="bf16"),
    "64": dict(rows=(2, 9), H=2, d=64, dtype="bf16", fused=True),
    "128": dict(rows=(3, 7), H=4, d=128, dtype="bf16"),
    "128-f32": dict(rows=(3, 7), H=4, d=128, dtype="f32", fused=True),
    "101": dict(rows=(11,), H=2, d=101, dtype="f32", fused=True),
    "256": dict(rows=(9,), H=3, d=256, dtype="bf16"),
    "250": dict(rows=(9,), H=3, d=250, dtype="bf16", fused=True),
    "512-f32": dict(rows=(5,), H=1, d=512, dtype="f32"),
    "1000": dict(rows=(4,), H=2, d=1000, dtype="bf16"),
    "2048": dict(rows=(3,), H=1, d=2048, dtype="bf16", fused=True),
    "2050": dict(rows=(3,), H=1, d=2050, dtype="f32"),
    "4096-f32": dict(rows=(2,), H=1, d=4096, dtype="f32"),
    "8191": dict(rows=(2,), H=1, d=8191, dtype="bf16"),
    "8192": dict(rows=(3,), H=1, d=8192, dtype="bf16"),
    "8192-f32": dict(rows=(2,), H=1, d=8192, dtype="f32"),
    "many-rows": dict(rows=(2, 4001), H=9, d=128, dtype="bf16"),
    "many-odd-rows": dict(rows=(30011,), H=1, d=31, dtype="f32"),
}


def gated_inputs(rows, H, d, dtype, fused=False, weight=True, seed=0):
    gen = torch.Generator().manual_seed(6000 + seed)
    dt = DT[dtype]
    x, z = (cut(gen, rows, H * d, dt, fused).unflatten(-1, (H, d)) for _ in "xz")
    w = (1 + 0.3 * torch.randn(d, generator=gen)).cuda() if weight else None
    z.mul_(3)
    return x, z, w, torch.randn(*rows, H, d, generator=gen).to(dt).cuda()


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("case", GATED)
def test_gated(case, act):
    x, z, w, dy = gated_inputs(**GATED[case])
    note(f"gated_norm {case} {act}")
    y = kda.gated_norm_forward(x, z, w, activation=act)
    g = kda.gated_norm_backward(x, z, dy, w, activation=act)
    torch.cuda.synchronize()
    ry, my = ref.gated(x, z, w, act)
    check("y", y, ry, my, N)
    rg, rm = ref.gated_grad(x, z, dy, w, act)
    for key in ("dx", "dgate"):
        check(key, g[key], rg[key], rm[key], N)
    check("dweight", g["dweight"], rg["dweight"], rm["dweight"], N + x[..., 0].numel())


def test_gated_without_weight():
    x, z, _, dy = gated_inputs((7,), 2, 64, "f32", weight=False, seed=1)
    note("gated_norm without weight")
    y = kda.gated_norm_forward(x, z)
    g = kda.gated_norm_backward(x, z, dy)
    assert g["dweight"] is None
    ry, my = ref.gated(x, z)
    check("y", y, ry, my, N)
    dw = torch.empty(64, device="cuda")
    g = kda.gated_norm_backward(x, z, dy, out=dict(dweight=dw))
    rg, rm = ref.gated_grad(x, z, dy)
    assert g["dweight"] is dw
    for key in ("dx", "dgate", "dweight"):
        check(key, g[key], rg[key], rm[key], N + 14)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gates_far_from_zero(act):
    """Gates of +-30 keep the relative accuracy of the small side, +-1e4 give 0 or 1 without a NaN."""
    x, z, w, dy = gated_inputs((6,), 1, 128, "f32", seed=2)
    z[0], z[1], z[2], z[3] = 30.0, -30.0, 1e4, -1e4
    note(f"gated_norm far gates {act}")
    y = kda.gated_norm_forward(x, z, w, activation=act)
    g = kda.gated_norm_backward(x, z, dy, w, activation=act)
    torch.cuda.synchronize()
    ry, my = ref.gated(x, z, w, act)
    check("y", y, ry, my, N)
    rg, rm = ref.gated_grad(x, z, dy, w, act)
    for key in ("dx", "dgate", "dweight"):
        check(key, g[key], rg[key], rm[key], N + 6)


# every way a row is spread, with and without scales and gradients of the sum
RESIDUAL = {
    "one": dict(rows=(1,), D=1, dtype="f32"),
    "odd": dict(rows=(5, 3), D=37, dtype="bf16", scale=0.5),
    "128": dict(rows=(3, 7), D=128, dtype="bf16", channels=True, fused=True),
    "200": dict(rows=(40,), D=200, dtype="f32", fused=True, scale=-2.0),
    "768": dict(rows=(17,), D=768, dtype="bf16", channels=True, scale=0.25),
    "1011": dict(rows=(9,), D=1011, dtype="f32", channels=True),
    "1024": dict(rows=(9,), D=1024, dtype="f32"),
    "2048": dict(rows=(2, 30), D=2048, dtype="bf16", channels=True),
    "4096": dict(rows=(7,), D=4096, dtype="bf16", fused=True),
    "4100": dict(rows=(3,), D=4100, dtype="bf16"),
    "8192": dict(rows=(3,), D=8192, dtype="bf16", channels=True),
    "8192-f32": dict(rows=(3,), D=8192, dtype="f32", channels=True, scale=3.0),
    "8189": dict(rows=(2,), D=8189, dtype="f32", channels=True),
    "many-rows": dict(rows=(9003,), D=256, dtype="bf16", channels=True),
    "many-wide-rows": dict(rows=(3001,), D=1024, dtype="f32"),
}


def residual_inputs(rows, D, dtype, channels=False, scale=1.0, fused=False, seed=0):
    gen = torch.Generator().manual_seed(7000 + seed)
    dt = DT[dtype]
    x, res = (cut(gen, rows, D, dt, fused) for _ in "xr")
    w = (1 + 0.3 * torch.randn(D, generator=gen)).cuda()
    c = torch.randn(D, generator=gen).cuda() if channels else None
    dy, dt_ = (torch.randn(*rows, D, generator=gen).to(dt).cuda() for _ in "yt")
    return x, res, w, dict(channel_scale=c, scale=scale), dy, dt_


@pytest.mark.parametrize("case", RESIDUAL)
def test_residual(case):
    x, res, w, kw, dy, dtotal = residual_inputs(**RESIDUAL[case])
    note(f"residual_norm {case}")
    y, total = kda.residual_norm_forward(x, res, w, **kw)
    c, scale = kw["channel_scale"], kw["scale"]
    torch.cuda.synchronize()
    ry, rt, my, mt = ref.residual(x, res, w, c, scale)
    check("y", y, ry, my, N)
    check("total", total, rt, mt, 4)
    rows = x[..., 0].numel()
    for with_total in (True, False):
        dt = dtotal if with_total else None
        g = kda.residual_norm_backward(x if c is not None else None, total, dy, dt, w, **kw)
        torch.cuda.synchronize()
        rg, rm = ref.residual_grad(x, total, dy, dt, w, c, scale)
        for key in ("dx", "dresidual"):
            check(key, g[key], rg[key], rm[key], N)
        check("dweight", g["dweight"], rg["dweight"], rm["dweight"], N + rows)
        if c is None:
            assert g["dchannel_scale"] is None and (g["dx"] is g["dresidual"]) == (scale == 1.0)
        else:
            check("dchannel_scale", g["dchannel_scale"], rg["dchannel_scale"], rm["dchannel_scale"], N + rows)


def test_residual_total_as_a_slice_and_outputs_given():
    x, res, w, kw, dy, dtotal = residual_inputs((6,), 64, "bf16", channels=True, seed=1)
    note("residual_norm outputs given")
    wide = torch.full((6, 70), 7.0, dtype=torch.bfloat16, device="cuda")
    y, total = kda.residual_norm_forward(x, res, w, **kw)
    wide[:, 3:67].copy_(total)
    dx = torch.empty_like(x)
    a = kda.residual_norm_backward(x, wide[:, 3:67], dy, dtotal, w, out=dict(dx=dx), **kw)
    b = kda.residual_norm_backward(x, total, dy, dtotal, w, **kw)
    assert a["dx"] is dx
    for key in a:
        assert torch.equal(a[key], b[key]), key
    plain = kda.residual_norm_backward(None, total, dy, dtotal, w, out=dict(dx=dx))
    assert plain["dx"] is dx and torch.equal(dx, plain["dresidual"])
    with pytest.raises(ValueError, match="needs x"):
        kda.residual_norm_backward(None, total, dy, dtotal, w, **kw)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row(value):
    x, z, w, dy = gated_inputs((40,), 3, 96, "bf16", seed=3)
    note(f"block norms {value}")
    y, g = kda.gated_norm_forward(x, z, w), kda.gated_norm_backward(x, z, dy, w)
    x2 = x.clone()
    x2[7, 1, 5] = value
    y2, g2 = kda.gated_norm_forward(x2, z, w), kda.gated_norm_backward(x2, z, dy, w)
    other = torch.ones_like(y, dtype=torch.bool)
    other[7, 1] = False
    for a, b in ((y, y2), (g["dx"], g2["dx"]), (g["dgate"], g2["dgate"])):
        assert torch.equal(a[other], b[other])
    assert not torch.isfinite(y2[7, 1, 5])
    r, t = kda.residual_norm_forward(x[:, 0], z[:, 0], w)
    r2, t2 = kda.residual_norm_forward(x2[:, 1], z[:, 1], w)
    assert torch.isfinite(r).all() and not torch.isfinite(r2[7]).all() and torch.isfinite(r2[:7]).all()
    assert torch.isfinite(t2[8:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small_rows_and_no_epsilon(dtype):
    """Rows of 1e15 (whose squares fit fp32) and 1e-15, and rows of zeros with the epsilon."""
    x, z, w, dy = gated_inputs((6,), 1, 128, dtype, seed=4)
    x[0] *= 1e15
    x[1] *= 1e-15
    x[2] = 0
    note("block norms large rows")
    y = kda.gated_norm_forward(x, z, w)
    ry, my = ref.gated(x, z, w)
    check("y", y, ry, my, N)
    x[2] = 1
    y = kda.gated_norm_forward(x, z, w, eps=0.0)
    g = kda.gated_norm_backward(x, z, dy, w, eps=0.0)
    ry, my = ref.gated(x, z, w, eps=0.0)
    check("y", y, ry, my, N)
    rg, rm = ref.gated_grad(x, z, dy, w, eps=0.0)
    for key in ("dx", "dgate", "dweight"):
        check(key, g[key], rg[key], rm[key], N + 6)


def test_autograd_and_determinism():
    x, z, w, dy = gated_inputs((2, 50), 4, 64, "bf16", seed=5)
    note("block norms autograd")
    leaves = [t.clone().requires_grad_() for t in (x, z, w)]
    kda.gated_norm(*leaves, activation="silu").backward(dy)
    g, again = (kda.gated_norm_backward(x, z, dy, w, activation="silu") for _ in "ab")
    for t, key in zip(leaves, ("dx", "dgate", "dweight")):
        assert torch.equal(t.grad, g[key]) and torch.equal(again[key], g[key]), key
    x, res, w, kw, dy, dtotal = residual_inputs((2, 30), 256, "f32", channels=True, seed=6)
    leaves = [t.clone().requires_grad_() for t in (x, res, w, kw["channel_scale"])]
    y, total = kda.residual_norm(*leaves[:3], channel_scale=leaves[3])
    torch.autograd.backward([y, total], [dy, dtotal])
    _, total = kda.residual_norm_forward(x, res, w, **kw)
    g, again = (kda.residual_norm_backward(x, total, dy, dtotal, w, **kw) for _ in "ab")
    for t, key in zip(leaves, ("dx", "dresidual", "dweight", "dchannel_scale")):
        assert torch.equal(t.grad, g[key]) and torch.equal(again[key], g[key]), key
    # only one of the two results used, and no scale: x's gradient is the sum's
    leaves = [t.clone().requires_grad_() for t in (x, res, w)]
    y, _ = kda.residual_norm(*leaves)
    y.backward(dy)
    assert torch.equal(leaves[0].grad, leaves[1].grad)
    _, total = kda.residual_norm_forward(x, res, w)
    assert torch.equal(leaves[1].grad, kda.residual_norm_backward(None, total, dy, None, w)["dresidual"])


def test_gradients_against_differences():
    """fp32 gradients along random directions against central differences of the 64-bit forward."""
    gen = torch.Generator().manual_seed(8)
    step = 1e-5
    x, z, w, dy = gated_inputs((7,), 2, 40, "f32", seed=7)
    note("block norms differences")
    g = kda.gated_norm_backward(x, z, dy, w)
    base = dict(x=x.double().cpu(), z=z.double().cpu(), w=w.double().cpu())
    of = dict(x="dx", z="dgate", w="dweight")

    def compare(f, base, of, g):
        for n, key in of.items():
            d = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
            diff = (f(dict(base, **{n: base[n] + step * d})) - f(dict(base, **{n: base[n] - step * d}))) / (2 * step)
            got = g[key].double().cpu()
            room = 200 * 2.0 ** -24 * float((got * d).abs().sum()) + 1e-6
            assert abs(float((got * d).sum()) - diff) <= room, key
    compare(lambda p: float((ref.gated(**p)[0] * dy.double().cpu()).sum()), base, of, g)
    x, res, w, kw, dy, dtotal = residual_inputs((7,), 40, "f32", channels=True, scale=0.5, seed=8)
    _, total = kda.residual_norm_forward(x, res, w, **kw)
    g = kda.residual_norm_backward(x, total, dy, dtotal, w, **kw)
    base = dict(x=x.double().cpu(), res=res.double().cpu(), w=w.double().cpu(), c=kw["channel_scale"].double().cpu())

    def f(p):
        y, t, _, _ = ref.residual(**p, scale=0.5)
        return float((y * dy.double().cpu()).sum() + (t * dtotal.double().cpu()).sum())
    compare(f, base, dict(x="dx", res="dresidual", w="dweight", c="dchannel_scale"), g)
