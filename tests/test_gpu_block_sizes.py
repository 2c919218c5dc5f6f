"""Linear attention over many slots (block_sizes.py) against its plain 64-bit
form, every element; tolerances as in test_gpu_linear_attn.py, whose state
part counts the slots (each is at least two chunks of 32 tokens)."""
import pytest
import torch

import block_reference as ref
import block_sizes
import gated_delta_rule_105_amd as kda
import test_gpu_linear_attn as linear
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", block_sizes.LINEAR)
def test_forward(name):
    c = block_sizes.case(name)
    p, cu, _ = linear.inputs(**c, seed=2)
    note(f"linear_attn_forward sizes {name}")
    o, ht = kda.linear_attn_forward(**p, cu_seqlens=cu)
    torch.cuda.synchronize()
    ro, rht, mo, mht = ref.linear(**p, cu=cu)
    check("o", o, ro, mo, linear.roundings(c))
    check("ht", ht, rht, mht, 300 * (linear.longest(c) // 32 + 2))


@pytest.mark.parametrize("name", [n for n in block_sizes.LINEAR if n != "two-packed"])
def test_backward(name):
    c = block_sizes.case(name)
    p, cu, u = linear.inputs(**c, seed=3)
    note(f"linear_attn_backward sizes {name}")
    g = kda.linear_attn_backward(**p, **u, cu_seqlens=cu)
    torch.cuda.synchronize()
    rg, rm = ref.linear_grad(**p, **u, cu=cu)
    n = linear.roundings(c)
    for key in ("dq", "dk", "dv", "dh0"):
        check(key, g[key], rg[key], rm[key], n)
    check("dg", g["dg"], rg["dg"], ref.suffix_magnitudes(**p, **u, cu=cu), n)

