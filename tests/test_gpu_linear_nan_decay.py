"""A NaN among the log decays of linear attention reaches what the recurrence
carries it to: outputs and dq of its own and later tokens, dk, dv and dh0 of
earlier ones, and nothing of another head or sequence."""
import pytest
import torch

import gated_delta_rule_105_amd as kda
import test_gpu_linear_attn as linear
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [50, 51, 120, 249])
@pytest.mark.parametrize("dk,dv", [(64, 64), (3, 5), (100, 128)])
@pytest.mark.parametrize("rows", [1, 130])
def test_nan_among_the_decays(at, dtype, dk, dv, rows):
    """Sequences of 50 and 200 tokens, or rows of 250 of which the first holds the NaN."""
    lengths = [50, 200, 40] if rows == 1 else None
    lo = 50 if lengths else 0
    p, cu, u = linear.inputs(rows, 250, 2, 2, dk, dv, dtype, lengths=lengths, seed=51)
    note(f"linear_attn NaN among decays {at} {dtype} {dk} {dv} {rows}")
    p["g"][0, at, 1] = float("nan")
    o, ht = kda.linear_attn_forward(**p, cu_seqlens=cu)
    g = kda.linear_attn_backward(**p, **u, cu_seqlens=cu)
    torch.cuda.synchronize()
    for name, t, span in (("o", o, slice(at, 250)), ("dq", g["dq"], slice(at, 250)), ("dk", g["dk"], slice(lo, at)),
                          ("dv", g["dv"], slice(lo, at))):
        hit = torch.zeros_like(t, dtype=torch.bool)
        hit[0, span, 1] = True
        wrong = (torch.isfinite(t) == hit).nonzero()
        assert wrong.numel() == 0, (name, wrong[0].tolist(), wrong[-1].tolist(), wrong.shape[0])
    for name, t in (("ht", ht), ("dh0", g["dh0"])):
        hit = torch.zeros_like(t, dtype=torch.bool)
        hit[1 if lengths else 0, 1] = True
        assert torch.equal(torch.isfinite(t), ~hit), name
    other = torch.ones_like(g["dg"], dtype=torch.bool)
    other[0, lo:250, 1] = False
    assert torch.isfinite(g["dg"][other]).all()
