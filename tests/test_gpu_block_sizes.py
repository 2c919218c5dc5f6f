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


@pytest.mark.parametrize("name", [n for n in block_sizes.LINEAR if n != "three-packed"])
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



def shifted(shape, dtype):
    """A contiguous tensor one element behind a vector's boundary, between elements that nothing may write."""
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + 2,), 7.0, dtype=dtype, device="cuda")
    return whole, whole[1:-1].view(shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 40, 7])
def test_outputs_and_gradients_at_single_elements(dtype, d):
    """What a call writes lies at any element, as its inputs do: bit for bit what it is elsewhere."""
    dt = linear.DT[dtype]
    p, cu, u = linear.inputs(B=2, T=70, Hq=2, H=2, dk=d, dv=d, dtype=dtype, seed=4)
    note(f"outputs at single elements {dtype} {d}")
    o, _ = kda.linear_attn_forward(**p)
    whole, odd = shifted(o.shape, dt)
    kda.linear_attn_forward(**p, o=odd)
    seen = [(whole, odd, o)]
    g = kda.linear_attn_backward(**p, **u)
    out = {k: shifted(g[k].shape, dt) for k in ("dq", "dk", "dv", "dg")}
    do_whole, do = shifted(o.shape, dt)
    do.copy_(u["do"])
    kda.linear_attn_backward(**p, do=do, dht=u["dht"], out={k: v[1] for k, v in out.items()})
    seen += [(*out[k], g[k]) for k in out] + [(do_whole, do, u["do"])]
    y = kda.gated_norm_forward(o, p["v"])
    whole, odd = shifted(y.shape, dt)
    kda.gated_norm_forward(o, p["v"], y=odd)
    seen.append((whole, odd, y))
    n = kda.gated_norm_backward(o, p["v"], u["do"])
    out = {k: shifted(n[k].shape, dt) for k in ("dx", "dgate")}
    kda.gated_norm_backward(o, p["v"], do, out={k: v[1] for k, v in out.items()})
    seen += [(*out[k], n[k]) for k in out]
    x, r = o.flatten(2), u["do"].flatten(2)
    y, total = kda.residual_norm_forward(x, r)
    a, b = shifted(y.shape, dt), shifted(y.shape, dt)
    kda.residual_norm_forward(x, r, y=a[1], total=b[1])
    seen += [(*a, y), (*b, total)]
    torch.cuda.synchronize()
    for whole, odd, want in seen:
        assert torch.equal(odd, want)
        assert whole[0] == 7.0 and whole[-1] == 7.0
