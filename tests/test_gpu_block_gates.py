"""The gates of the gated norm far from zero, in fp32 against 64 bits: an
exponential of z whose argument is rounded would be |z| roundings off.

x is one channel, so that its norm is its sign and y = act(z).  Roundings of
y: the norm's root, quotient and product (1.5 together: each at most half a
step of a value up to 1, which is 1 times 2^-24), the exponential within 3,
1 + e^-z 1, its reciprocal 2 and one product 1 each with the norm, the weight
and SiLU's z: below 10 times 2^-24.  The slopes are sums of two such terms of
SiLU, and e / (1 + e)^2 of the sigmoid: below 16 of the terms' magnitudes.
"""
import pytest
import torch

import gated_delta_rule_105_amd as kda
from gpu_util import note

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gates_far_from_zero(act):
    note(f"gates far from zero {act}")
    gen = torch.Generator().manual_seed(1)
    z = torch.cat([torch.linspace(-86.0, 86.0, 20001), 3 * torch.randn(20000, generator=gen)])[:, None, None]
    x = torch.ones_like(z)
    y = kda.gated_norm_forward(x.cuda(), z.cuda(), activation=act, eps=0.0).cpu().double()
    one = torch.ones(1, device="cuda")
    r = kda.gated_norm_backward(x.cuda(), z.cuda(), x.cuda(), one, activation=act, eps=0.0)
    dgate = r["dgate"].cpu().double()
    z = z.double()
    s, c = torch.sigmoid(z), torch.sigmoid(-z)
    a = s if act == "sigmoid" else z * s
    slope = s * c if act == "sigmoid" else s + z * s * c
    terms = s * c if act == "sigmoid" else s + (z * s * c).abs()
    assert float(((y - a).abs() / (a.abs() + 1e-37)).max()) <= 10 * ULP
    assert float(((dgate - slope).abs() / (terms + 1e-37)).max()) <= 16 * ULP
    assert abs(float(r["dweight"][0]) / float(a.sum()) - 1) <= 1e-5
