"""The operators around the recurrence at the sizes of layer_sizes.py, against
the plain 64-bit forms, every element.  Roundings as derived in
test_gpu_short_conv.py, test_gpu_selective_scan.py and test_gpu_qk_norm.py."""
import pytest
import torch

import gated_delta_rule_105_amd as kda
import layer_reference as ref
import layer_sizes
import test_gpu_qk_norm as norm_cases
import test_gpu_selective_scan as scan_cases
import test_gpu_short_conv as conv_cases
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", layer_sizes.CONV)
def test_convolution(case):
    c = layer_sizes.CONV[case]
    p = conv_cases.inputs(c.get("B", 1), c.get("T", 0), c["D"], c["W"], c["dtype"], lengths=c.get("lengths"), seed=20)
    dev = conv_cases.dev
    note(f"short_conv sizes {case}")
    kw = dict(initial_state=dev(p["init"]), cu_seqlens=dev(p["cu"]), activation=c["act"])
    y, fin = kda.short_conv_forward(dev(p["x"]), dev(p["w"]), dev(p["bias"]), **kw)
    g = kda.short_conv_backward(dev(p["x"]), dev(p["w"]), dev(p["dy"]), dev(p["bias"]), dfinal=dev(p["dfinal"]), **kw)
    torch.cuda.synchronize()
    ry, rf, my = ref.conv(p["x"], p["w"], p["bias"], p["init"], p["cu"], c["act"])
    check("y", y, ry, my, 64)
    assert torch.equal(fin.cpu().double(), rf)
    rg, rm = ref.conv_grad(p["x"], p["w"], p["dy"], p["bias"], p["init"], p["dfinal"], p["cu"], c["act"])
    n = p["x"].shape[0] * p["x"].shape[1]
    for key, r in (("dx", 128), ("dweight", 128 + n), ("dbias", 128 + n), ("dinitial", 128)):
        check(key, g[key], rg[key], rm[key], r)


@pytest.mark.parametrize("case", layer_sizes.SCAN)
def test_scan(case):
    c = {k: v for k, v in layer_sizes.SCAN[case].items() if k not in ("slots", "carry")}
    p, q, u, _ = scan_cases.inputs(**c, seed=21)
    note(f"selective_scan sizes {case}")
    o, ht = kda.selective_scan_forward(**p, **q)
    g = kda.selective_scan_backward(**p, **q, **u)
    torch.cuda.synchronize()
    longest = scan_cases.longest(c)
    ro, rht, mo, mht = ref.scan(**p, h0=q["h0"], cu=q["cu_seqlens"])
    check("o", o, ro, mo, 64 + 8 * longest)
    check("ht", ht, rht, mht, 64 + 8 * longest)
    rg, rm = ref.scan_grad(**p, **u, h0=q["h0"], cu=q["cu_seqlens"])
    n, tokens = 128 + 16 * longest, p["x"].shape[0] * p["x"].shape[1]
    for key in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"):
        check(key, g[key], rg[key], rm[key], n + (tokens if key in ("dA", "dD", "ddt_bias") else 0))


@pytest.mark.parametrize("case", layer_sizes.STEP)
def test_scan_step(case):
    c = layer_sizes.STEP[case]
    p, q, _, _ = scan_cases.inputs(c["S"], 2, c["D"], c["N"], c["dtype"], G=c["G"], fused=True, seed=22)
    note(f"selective_scan_step sizes {case}")
    ro, rht, mo, mht = ref.scan(**p, h0=q["h0"])
    state = q["h0"].clone()
    for t in range(2):
        tok = {k: (v[:, t] if k in ("x", "dt", "z", "B", "C") else v) for k, v in p.items()}
        o = kda.selective_scan_step(state=state, **tok)
        torch.cuda.synchronize()
        check("o", o, ro[:, t], mo[:, t], 64 + 16)
    check("state", state, rht, mht, 64 + 16)


@pytest.mark.parametrize("kind,inter,scale", norm_cases.KINDS)
@pytest.mark.parametrize("case", layer_sizes.NORM)
def test_norm(case, kind, inter, scale):
    c = {k: v for k, v in layer_sizes.NORM[case].items() if k not in ("steps", "waves")}
    p = norm_cases.inputs(**c, fused=True, seed=23)
    note(f"qk_norm sizes {case} {kind}")
    opt = norm_cases.options(kind, inter, scale)
    args = (p["wq"], p["wk"], p["pos"], p["freq"])
    q, k = kda.qk_norm_forward(p["q"], p["k"], *args, **opt)
    g = kda.qk_norm_backward(p["q"], p["k"], p["dq"], p["dk"], *args, **opt)
    torch.cuda.synchronize()
    for n, out, x, w, s, d in (("q", q, p["q"], p["wq"], scale, p["dq"]), ("k", k, p["k"], p["wk"], 1.0, p["dk"])):
        check(n, out, *ref.norm(x, w, p["pos"], p["freq"], kind, 1e-5, inter, s), 64)
        dx, dw, mx, mw = ref.norm_grad(x, d, w, p["pos"], p["freq"], kind, 1e-5, inter, s)
        check("d" + n, g["d" + n], dx, mx, 128)
        check(f"d{n}_weight", g[f"d{n}_weight"], dw, mw, 128 + x.numel() // x.shape[-1])


def test_nan_stays_in_its_channel_beside_padding():
    """States past N (12 of 16) and channels past D: a NaN changes no other channel by a bit."""
    p, q, u, _ = scan_cases.inputs(1, 0, 37, 12, "f32", lengths=[50, 300, 43], seed=24)
    note("selective_scan nan beside padding")
    o, ht = kda.selective_scan_forward(**p, **q)
    g = kda.selective_scan_backward(**p, **q, **u)
    p2 = dict(p, x=p["x"].clone())
    p2["x"][0, 200, 7] = float("nan")
    o2, ht2 = kda.selective_scan_forward(**p2, **q)
    g2 = kda.selective_scan_backward(**p2, **q, **u)
    torch.cuda.synchronize()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 200:350, 7] = True
    assert torch.equal(torch.isnan(o2), hit) and torch.equal(o2[~hit], o[~hit])
    hit = torch.zeros_like(ht, dtype=torch.bool)
    hit[1, 7] = True
    assert torch.equal(torch.isnan(ht2), hit) and torch.equal(ht2[~hit], ht[~hit])
    for key in ("dx", "ddt", "dz"):
        other = torch.ones(g[key].shape, dtype=torch.bool, device="cuda")
        other[0, 50:350, 7] = False
        assert torch.equal(g2[key][other], g[key][other]), key
    for key in ("dB", "dC"):
        assert torch.equal(g2[key][0, :200], g[key][0, :200]) and torch.equal(g2[key][0, 350:], g[key][0, 350:]), key
    for key in ("dA", "dD", "ddt_bias"):
        other = torch.arange(37, device="cuda") != 7
        assert torch.equal(g2[key][other], g[key][other]), key
