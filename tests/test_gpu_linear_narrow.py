"""Linear attention with fewer channels than a 16-byte vector holds, over
several chunks: against the plain 64-bit form, tolerances as in
test_gpu_linear_attn.py, and infinities among such channels.

That these heads go through by chunks shows in test_gpu_linear_state.py: token
by token the state would take a rounding for each token.
"""
import pytest
import torch

import block_reference as ref
import gated_delta_rule_105_amd as kda
import test_gpu_linear_attn as linear
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu
DIMS = [(1, 1), (3, 7), (7, 3), (1, 64), (64, 1), (2, 100), (100, 2)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [dict(B=2, T=150), dict(B=64, T=70), dict(B=1, T=0, lengths=[130, 0, 1, 90])])
def test_narrow_heads(rows, dtype, dk, dv):
    c = dict(rows, Hq=2, H=4, dk=dk, dv=dv, dtype=dtype)
    p, cu, u = linear.inputs(**c, seed=21, fused=dtype == "bf16")
    note(f"linear_attn narrow {rows} {dtype} {dk} {dv}")
    o, ht = kda.linear_attn_forward(**p, cu_seqlens=cu)
    g = kda.linear_attn_backward(**p, **u, cu_seqlens=cu)
    torch.cuda.synchronize()
    n = linear.roundings(c)
    ro, rht, mo, mht = ref.linear(**p, cu=cu)
    check("o", o, ro, mo, n)
    check("ht", ht, rht, mht, 300 * (linear.longest(c) // 32 + 2))
    rg, rm = ref.linear_grad(**p, **u, cu=cu)
    for key in ("dq", "dk", "dv", "dh0"):
        check(key, g[key], rg[key], rm[key], n)
    check("dg", g["dg"], rg["dg"], ref.suffix_magnitudes(**p, **u, cu=cu), n)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_among_narrow_values(value, dtype):
    """What is not finite in the second chunk reaches later tokens of its column, nothing else."""
    p, _, u = linear.inputs(1, 200, 1, 2, 3, 3, dtype, seed=22)
    note(f"linear_attn narrow {value} {dtype}")
    o, _ = kda.linear_attn_forward(**p)
    v = p["v"].clone()
    v[0, 100, 1, 2] = value
    o2, ht2 = kda.linear_attn_forward(**dict(p, v=v))
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 100:, 1, 2] = True
    assert torch.equal(torch.isfinite(o2), ~hit)
    hit_h = torch.zeros_like(ht2, dtype=torch.bool)
    hit_h[0, 1, :, 2] = True
    assert torch.equal(torch.isfinite(ht2), ~hit_h)
    do = u["do"].clone()
    do[0, 100, 1, 2] = value
    g = kda.linear_attn_backward(**p, **dict(u, do=do))
    hit = torch.zeros_like(g["dv"], dtype=torch.bool)
    hit[0, :101, 1, 2] = True
    assert torch.equal(torch.isfinite(g["dv"]), ~hit)
    q = p["q"].clone()
    q[0, 100, 0, 1] = value
    g = kda.linear_attn_backward(**dict(p, q=q), **u)
    hit = torch.zeros_like(g["dk"], dtype=torch.bool)
    hit[0, :101, :, 1] = True
    assert torch.equal(torch.isfinite(g["dk"]), ~hit)
