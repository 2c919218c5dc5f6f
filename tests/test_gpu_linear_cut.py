"""Log decays whose factor is 0 in linear attention's gradients: nothing passes
such a token, so its own gradient is 0 and what follows it does not reach the
gradients before it, not even as a rounding."""
import pytest
import torch

import block_reference as ref
import gated_delta_rule_105_amd as kda
import test_gpu_linear_attn as linear
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low", [float("-inf"), -88.0, -3e4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [dict(B=2, T=300), dict(B=128, T=150), dict(B=1, T=0, lengths=[140, 0, 1, 160])])
def test_nothing_passes(shape, dtype, low):
    c = dict(shape, Hq=2, H=2, dk=64, dv=64, dtype=dtype)
    p, cu, u = linear.inputs(**c, seed=31)
    note(f"linear_attn cut {shape} {dtype} {low}")
    at = [3, 4, 70, 127]
    p["g"][:, at, 1] = low
    one = kda.linear_attn_backward(**p, **u, cu_seqlens=cu)["dg"]
    assert (one[:, at, 1] == 0).all()
    assert (one[:, :128, 0] != 0).any(1).all()
    # other gradients of the tokens from the last cut on, as large as they come
    do = u["do"].clone()
    do[:, 127:140] *= 1000.0
    v = p["v"].clone()
    v[:, 127:140] *= 1000.0
    two = kda.linear_attn_backward(**dict(p, v=v), **dict(u, do=do), cu_seqlens=cu)["dg"]
    torch.cuda.synchronize()
    assert torch.equal(one[:, :127, 1], two[:, :127, 1])
    rows = slice(0, 2) if c["B"] > 2 else slice(None)
    few = {k: x[rows] if x is not None and k not in ("scale",) else x for k, x in p.items()}
    us = {k: x[rows] if cu is None else x for k, x in u.items()}
    few["h0"] = p["h0"][rows] if cu is None else p["h0"]
    want, _ = ref.linear_grad(**few, **us, cu=cu)
    check("dg", one[rows], want["dg"], ref.suffix_magnitudes(**few, **us, cu=cu), linear.roundings(c))
