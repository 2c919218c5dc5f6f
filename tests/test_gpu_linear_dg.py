"""The gradients of linear attention, every element, within the bounds of
linear_dg.py, of which test_linear_dg_bounds.py shows that the decays' reject
wrong sums."""
import pytest
import torch

import gated_delta_rule_105_amd as kda
import linear_dg
import test_gpu_linear_attn as linear
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", linear_dg.CASES)
def test_gradients(name):
    p, cu, u, rows = linear_dg.inputs(name, linear.inputs)
    note(f"linear_attn dg {name}")
    got = kda.linear_attn_backward(**p, **u, cu_seqlens=cu)
    dtype = p["q"].dtype
    if rows:
        p, u = linear_dg.first(rows, p, u)
    for key, (want, room) in linear_dg.bounds(p, u, cu, dtype).items():
        if got[key] is None:
            continue
        off = (got[key].cpu().double()[:rows] - want).abs() / room
        assert float(off.max()) <= 1, (key, float(off.max()), int((off > 1).sum()), off.numel())
        print(f"{name} {key}: at most {float(off.max()):.3f} of the bound")
