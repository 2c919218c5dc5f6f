"""What linear attention's products keep of 32-bit weights, states and decayed
values: sums in which all but the last bits cancel, exactly as in 64 bits.

Every number below is a sum of few powers of two and every partial sum has
fewer than 24 bits, so arithmetic in 32 bits makes no rounding at all: outputs
are the 64-bit values, rounded once to the outputs' type.  A weight, state or
value that is read with 17 bits loses the part of 2^-18 that is all there is.
"""
import pytest
import torch

import block_reference as ref
import gated_delta_rule_105_amd as kda
from gpu_util import note

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DIMS = [(64, 64), (128, 128), (64, 128), (128, 64), (20, 9)]
LONG, SHORT = (1.0, 2.0 ** -9, 2.0 ** -18), (1.0, 2.0 ** -9, 0.0)
ROWS = [(1, 90), (256, 40)]  # in slots; rows that fill the device


def zeros(B, T, dk, dv, dtype):
    shape = lambda d: torch.zeros(B, T, 1, d, dtype=DT[dtype], device="cuda")  # noqa: E731
    return dict(q=shape(dk), k=shape(dk), v=shape(dv), do=shape(dv))


def alternate(weights, values):
    """Tokens whose weights are 1 + 2^-9 + 2^-18 and 1 + 2^-9 in turn, whose values 1 and -1."""
    for i, w in enumerate(LONG):
        weights[:, 0::2, :, i] = w
    for i, w in enumerate(SHORT):
        weights[:, 1::2, :, i] = w
    values[:, 0::2] = 1.0
    values[:, 1::2] = -1.0


def same(name, got, want):
    """got is want rounded once; rows of a batch are all alike."""
    assert torch.equal(got[:1].cpu(), want[:1].to(got.dtype)), name
    assert torch.equal(got, got[:1].expand_as(got)), name


def run(x, h0=None, dht=None, g=None):
    """o, ht and gradients, and the same of one row in 64 bits."""
    p = dict(q=x["q"], k=x["k"], v=x["v"], g=g, h0=h0)
    o, ht = kda.linear_attn_forward(**p)
    got = dict(kda.linear_attn_backward(**p, do=x["do"], dht=dht), o=o)
    one = {n: t[:1] if t is not None else None for n, t in dict(p, do=x["do"], dht=dht).items()}
    want, _ = ref.linear_grad(**one)
    del one["do"], one["dht"]
    want["o"] = ref.linear(**one)[0]
    torch.cuda.synchronize()
    return got, want


@pytest.mark.parametrize("B,T", ROWS)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["o", "dq", "dk", "dv"])
def test_weights(out, dtype, dk, dv, B, T):
    note(f"linear_attn bits of weights {out} {dtype} {dk} {dv} {B}")
    x = zeros(B, T, dk, dv, dtype)
    # the operand whose products with the other's rows are the weights, and what they weight
    ones, weights, values = {"o": ("q", "k", "v"), "dv": ("k", "q", "do"), "dq": ("do", "v", "k"),
                             "dk": ("v", "do", "q")}[out]
    x[ones][..., :3] = 1.0
    alternate(x[weights], x[values])
    got, want = run(x)
    assert want[out].abs().max() > 0 and 0 < want[out][want[out] != 0].abs().min() <= 2.0 ** -17
    same(out, got[out], want[out])


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["o", "dq", "dk", "dv"])
def test_states(out, dtype, dk, dv):
    note(f"linear_attn bits of states {out} {dtype} {dk} {dv}")
    x = zeros(2, 70, dk, dv, dtype)
    state = torch.zeros(2, 1, dk, dv, device="cuda")
    of_keys = out in ("o", "dv")  # sums over the state's rows
    rows = state if of_keys else state.transpose(2, 3)
    rows[:, :, 0] = 1 + 2.0 ** -9 + 2.0 ** -18
    rows[:, :, 1] = 1 + 2.0 ** -9
    meets = x[{"o": "q", "dq": "do", "dk": "v", "dv": "k"}[out]]
    meets[..., 0], meets[..., 1] = 1.0, -1.0
    got, want = run(x, **{"h0" if out in ("o", "dq") else "dht": state})
    assert (want[out] == 2.0 ** -18).any()
    same(out, got[out], want[out])


@pytest.mark.parametrize("B,T", [(1, 128), (2, 700), (256, 128)])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decayed_values(dtype, dk, dv, B, T):
    """A token that adds what its sequence's first state has become (or, back in time, its last gradient): nothing is
    left of either, whatever the decay."""
    note(f"linear_attn bits of decayed values {dtype} {dk} {dv} {B}")
    gen = torch.Generator().manual_seed(3)
    g = (-0.05 * torch.rand(1, T, 1, generator=gen)).to(DT[dtype]).cuda().expand(B, T, 1).contiguous()
    g[:, 0] = 0.0
    x = zeros(B, T, dk, dv, dtype)
    minus = torch.full((B, 1, dk, dv), -1.0, device="cuda")
    # forward: the first token's k v^T is what h0 is not
    x["k"][:, 0], x["v"][:, 0] = 1.0, 1.0
    x["q"][:, 1:], x["do"][:, 1:] = 1.0, 1.0
    got, _ = run(x, h0=minus, g=g)
    for key in ("o", "dq"):
        assert (got[key] == 0).all(), key
    # back in time: the last token's q do^T is what dht is not
    x = zeros(B, T, dk, dv, dtype)
    x["q"][:, -1], x["do"][:, -1] = 1.0, 1.0
    x["k"][:, :-1], x["v"][:, :-1] = 1.0, 1.0
    got, _ = run(x, dht=minus, g=g)
    for key in ("dk", "dv"):
        assert (got[key][:, :-1] == 0).all(), key
