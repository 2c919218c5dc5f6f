"""Norm of queries and keys with the rotation against its plain 64-bit form,
every element.

Tolerance (layer_reference.check): half a step of the output's type plus fp32
roundings (2^-24) of the magnitudes.  A head's sum of squares has at most
d / 64 additions a lane and 6 between lanes, all of positive terms; root and
division a rounding each; norm, weight, scale and rotation under 12 more, the
cosine and the sine 4 each: under 64 in all for d up to 512.  The gradient
has two such sums (128), a weight's gradient one rounding per head summed.
"""
import pytest
import torch

import gated_delta_rule_105_amd as kda
import layer_reference as ref
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(rows, Hq, Hk, d, rot, dtype, weight=True, far=0, fused=False, seed=0):
    g = torch.Generator().manual_seed(2000 + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DT[dtype]
    if fused:
        whole = r(*rows, (Hq + 2 * Hk) * d + 1).to(dt).cuda()
        q = whole[..., 1: 1 + Hq * d].unflatten(-1, (Hq, d))
        k = whole[..., 1 + Hq * d: 1 + (Hq + Hk) * d].unflatten(-1, (Hk, d))
    else:
        q, k = r(*rows, Hq, d).to(dt).cuda(), r(*rows, Hk, d).to(dt).cuda()
    p = dict(q=q, k=k, wq=None, wk=None, pos=None, freq=None, dq=r(*rows, Hq, d).to(dt).cuda(),
             dk=r(*rows, Hk, d).to(dt).cuda())
    if weight:
        p["wq"], p["wk"] = r(d).cuda(), r(d).cuda()
    if rot:
        p["pos"] = torch.randint(far, far + 100, rows, generator=g).to(torch.int32).cuda()
        p["freq"] = (10000.0 ** (-torch.arange(0, rot, 2).float() / rot)).cuda()
    return p


# rows of tokens, heads, d, rotated channels
CASES = {
    "one-token": dict(rows=(1, 1), Hq=1, Hk=1, d=128, rot=128, dtype="bf16"),
    "unit-no-rotation": dict(rows=(2, 33), Hq=4, Hk=4, d=128, rot=0, dtype="bf16", weight=False),
    "decode": dict(rows=(5,), Hq=16, Hk=2, d=64, rot=64, dtype="bf16"),
    "partly-rotated-far": dict(rows=(1, 70), Hq=8, Hk=2, d=128, rot=64, dtype="bf16", far=1000000),
    "far-f32": dict(rows=(1, 40), Hq=3, Hk=1, d=64, rot=64, dtype="f32", far=2 ** 31 - 200),
    "negative-positions": dict(rows=(6,), Hq=2, Hk=2, d=32, rot=32, dtype="f32", far=-50),
    "smallest-head": dict(rows=(3, 5), Hq=3, Hk=2, d=2, rot=2, dtype="f32"),
    "odd-pairs": dict(rows=(1, 31), Hq=5, Hk=3, d=74, rot=38, dtype="bf16"),
    "single-pairs-wide": dict(rows=(1, 9), Hq=3, Hk=1, d=250, rot=250, dtype="f32"),
    "single-pairs-widest": dict(rows=(1, 9), Hq=2, Hk=2, d=510, rot=6, dtype="bf16"),
    "widest": dict(rows=(1, 17), Hq=2, Hk=1, d=512, rot=512, dtype="bf16"),
    "d256": dict(rows=(1, 17), Hq=2, Hk=2, d=256, rot=128, dtype="f32"),
    "d24": dict(rows=(1, 50), Hq=7, Hk=3, d=24, rot=8, dtype="bf16"),
    "many-heads": dict(rows=(1, 19), Hq=65, Hk=9, d=16, rot=16, dtype="f32", weight=False),
    "slice": dict(rows=(2, 41), Hq=6, Hk=2, d=64, rot=64, dtype="bf16", fused=True),
    "slice-odd": dict(rows=(1, 20), Hq=3, Hk=1, d=38, rot=0, dtype="f32", fused=True),
    "many-tokens": dict(rows=(2, 3000), Hq=2, Hk=1, d=64, rot=32, dtype="f32"),
}
KINDS = [("l2", False, 1.0), ("rms", True, 0.088)]


def options(kind, inter, scale):
    return dict(norm=kind, interleaved=inter, q_scale=scale, eps=1e-5)


@pytest.mark.parametrize("kind,inter,scale", KINDS)
@pytest.mark.parametrize("case", CASES)
def test_forward(case, kind, inter, scale):
    p = inputs(**CASES[case])
    note(f"qk_norm_forward {case} {kind}")
    q, k = kda.qk_norm_forward(p["q"], p["k"], p["wq"], p["wk"], p["pos"], p["freq"], **options(kind, inter, scale))
    torch.cuda.synchronize()
    for name, out, x, w, s in (("q", q, p["q"], p["wq"], scale), ("k", k, p["k"], p["wk"], 1.0)):
        assert out.is_contiguous()
        check(name, out, *ref.norm(x, w, p["pos"], p["freq"], kind, 1e-5, inter, s), 64)


@pytest.mark.parametrize("kind,inter,scale", KINDS)
@pytest.mark.parametrize("case", CASES)
def test_backward(case, kind, inter, scale):
    p = inputs(**CASES[case], seed=1)
    note(f"qk_norm_backward {case} {kind}")
    g = kda.qk_norm_backward(p["q"], p["k"], p["dq"], p["dk"], p["wq"], p["wk"], p["pos"], p["freq"],
                             **options(kind, inter, scale))
    torch.cuda.synchronize()
    for n, x, w, s, d in (("q", p["q"], p["wq"], scale, p["dq"]), ("k", p["k"], p["wk"], 1.0, p["dk"])):
        dx, dw, mx, mw = ref.norm_grad(x, d, w, p["pos"], p["freq"], kind, 1e-5, inter, s)
        check("d" + n, g["d" + n], dx, mx, 128)
        if w is None:
            assert g[f"d{n}_weight"] is None
        else:
            check(f"d{n}_weight", g[f"d{n}_weight"], dw, mw, 128 + x.numel() // x.shape[-1])


def test_rows_of_zeros_and_large_values():
    """A head of zeros stays zero (eps keeps the norm finite); heads of 1e18 keep their direction."""
    note("qk_norm zeros")
    q = torch.zeros(2, 3, 2, 64, device="cuda")
    q[0, 1, 1] = 1e18
    q[1, 2, 0] = -1e-18
    out, _ = kda.qk_norm_forward(q, q)
    torch.cuda.synchronize()
    ro, m = ref.norm(q)
    check("q", out, ro, m, 64)
    assert not out[0, 0].any()
    g = kda.qk_norm_backward(q, q, torch.ones_like(q), torch.ones_like(q))
    torch.cuda.synchronize()
    dx, _, mx, _ = ref.norm_grad(q, torch.ones_like(q))
    check("dq", g["dq"], dx, mx, 128)


def test_nan_stays_in_its_head():
    p = inputs((1, 30), 4, 2, 64, 64, "f32", seed=2)
    note("qk_norm nan")
    args = (p["wq"], p["wk"], p["pos"], p["freq"])
    q, k = kda.qk_norm_forward(p["q"], p["k"], *args)
    q2 = p["q"].clone()
    q2[0, 7, 2, 33] = float("nan")
    o, ok = kda.qk_norm_forward(q2, p["k"], *args)
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[0, 7, 2] = True
    assert torch.equal(torch.isnan(o), hit) and torch.equal(o[~hit], q[~hit]) and torch.equal(ok, k)


def test_autograd_and_weight_gradients_on_request():
    p = inputs((2, 21), 4, 2, 32, 16, "f32", seed=3)
    note("qk_norm autograd")
    leaves = {n: p[n].clone().requires_grad_() for n in ("q", "k", "wq", "wk")}
    q, k = kda.qk_norm(leaves["q"], leaves["k"], leaves["wq"], leaves["wk"], p["pos"], p["freq"], norm="rms")
    ((q * p["dq"]).sum() + (k * p["dk"]).sum()).backward()
    g = kda.qk_norm_backward(p["q"], p["k"], p["dq"], p["dk"], p["wq"], p["wk"], p["pos"], p["freq"], norm="rms")
    for a, b in (("q", "dq"), ("k", "dk"), ("wq", "dq_weight"), ("wk", "dk_weight")):
        assert torch.equal(leaves[a].grad, g[b]), a
    out = dict(dk_weight=torch.empty(32, device="cuda"))
    g = kda.qk_norm_backward(p["q"], p["k"], p["dq"], p["dk"], out=out)
    torch.cuda.synchronize()
    assert g["dq_weight"] is None
    _, dw, _, mw = ref.norm_grad(p["k"], p["dk"])
    check("dk_weight", g["dk_weight"], dw, mw, 128 + 84)
    # only k used
    k = p["k"].clone().requires_grad_()
    kda.qk_norm(p["q"], k)[1].sum().backward()
    assert torch.equal(k.grad, kda.qk_norm_backward(p["q"], p["k"], torch.zeros_like(p["q"]),
                                                    torch.ones_like(p["k"]))["dk"])
