"""The operators around the recurrence at values where padding, composed
decays or bookkeeping could show: no epsilon, growing states, infinities next
to lanes that have no state or channel, rows behind the last sequence, states
that are updated in place while a gradient still needs them."""
import pytest
import torch

import gated_delta_rule_105_amd as kda
import layer_reference as ref
import test_gpu_qk_norm as norm_cases
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norm without an epsilon
@pytest.mark.parametrize("Hq,Hk,d,rot", [(3, 1, 128, 0), (5, 4, 64, 64), (3, 1, 34, 34), (5, 1, 32, 16), (1, 1, 512, 0)])
@pytest.mark.parametrize("kind", ["l2", "rms"])
def test_norm_gradient_without_epsilon(Hq, Hk, d, rot, kind):
    """eps = 0 is allowed; the lanes of a wave beyond the last head, whose norm would be zero, add nothing to the
    weights' gradients.  Roundings as in test_gpu_qk_norm."""
    p = norm_cases.inputs((2, 23), Hq, Hk, d, rot, "f32", seed=40)
    note(f"qk_norm_backward eps 0 Hq={Hq} Hk={Hk} d={d} {kind}")
    g = kda.qk_norm_backward(p["q"], p["k"], p["dq"], p["dk"], p["wq"], p["wk"], p["pos"], p["freq"], norm=kind, eps=0.0)
    torch.cuda.synchronize()
    for n, x, w, dout in (("q", p["q"], p["wq"], p["dq"]), ("k", p["k"], p["wk"], p["dk"])):
        dx, dw, mx, mw = ref.norm_grad(x, dout, w, p["pos"], p["freq"], kind, 0.0)
        check("d" + n, g["d" + n], dx, mx, 128)
        check(f"d{n}_weight", g[f"d{n}_weight"], dw, mw, 128 + x.numel() // d)
