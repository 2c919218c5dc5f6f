"""The state of linear attention over long rows: its roundings must not grow
with the number of products or lie all to one side.

Every chunk multiplies the state by one decay and adds one sum.  In fp32 that
is a rounding of at most 1.3 times 2^-24 (the decay's) and one of at most 1 of
the state a chunk, independent from chunk to chunk where the inputs differ, so
that after n chunks the error's mean square over many states is at most
n (1.3^2 + 1) (2^-24 |S|)^2 with |S| the largest that the state has been.
Errors of one side would add up to n times their mean, and a state to which
products are added one by one takes a rounding for each.
"""
import pytest
import torch

import gated_delta_rule_105_amd as kda
from gpu_util import note

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


@pytest.mark.parametrize("d_k,d_v", [(4, 8), (4, 3), (2, 8)])
def test_state_that_only_decays(d_k, d_v):
    B, T, H, chunk = 16, 8192, 16, 32
    note(f"linear_attn state that only decays {d_k} {d_v}")
    gen = torch.Generator().manual_seed(11)
    g = -2e-3 * torch.rand(B, T, H, generator=gen)
    zero = torch.zeros(B, T, H, d_k, device="cuda")
    v = torch.zeros(B, T, H, d_v, device="cuda")
    one = torch.ones(B, H, d_k, d_v, device="cuda")
    o, ht = kda.linear_attn_forward(zero, zero, v, g.cuda(), h0=one)
    r = kda.linear_attn_backward(zero, zero, v, v, g.cuda(), h0=one, dht=one)
    torch.cuda.synchronize()
    want = torch.exp(g.double().sum(1))[..., None, None]
    for name, got in (("ht", ht), ("dh0", r["dh0"])):
        off = (got.cpu().double() / want - 1) / STEP
        assert float(off.square().mean()) <= T // chunk * (1.3 ** 2 + 1), name


def test_steps_that_only_decay():
    """The same by single tokens: a decay and a product of each."""
    N, H, T = 16, 16, 4096
    note("linear_attn_step that only decays")
    gen = torch.Generator().manual_seed(12)
    g = -2e-3 * torch.rand(T, N, H, generator=gen)
    zero = torch.zeros(N, H, 4, device="cuda")
    state = torch.ones(N, H, 4, 4, device="cuda")
    on_device = g.cuda()
    for t in range(T):
        kda.linear_attn_step(zero, zero, zero, state, on_device[t])
    torch.cuda.synchronize()
    off = (state.cpu().double() / torch.exp(g.double().sum(0))[..., None, None] - 1) / STEP
    assert float(off.square().mean()) <= T * (1.3 ** 2 + 1)


def test_state_that_only_grows():
    """Without a decay the state is a sum of T / 32 chunks' sums, each less than sqrt(32) of its own size beside it:
    the state's roundings are one a chunk."""
    B, T, H, d = 16, 8192, 16, 8
    note("linear_attn state that only grows")
    gen = torch.Generator().manual_seed(13)
    k = (1 + torch.rand(B, T, H, d, generator=gen)).cuda()
    v = (1 + torch.rand(B, T, H, d, generator=gen)).cuda()
    q = torch.zeros_like(k)
    o, ht = kda.linear_attn_forward(q, k, v)
    r = kda.linear_attn_backward(k, q, v, v, h0=torch.zeros_like(ht))  # dh0: sum q do^T
    torch.cuda.synchronize()
    want = k.double().permute(0, 2, 3, 1) @ v.double().permute(0, 2, 1, 3)
    n = T // 32
    for name, got in (("ht", ht), ("dh0", r["dh0"])):
        off = (got.double() / want - 1) / STEP
        # the state of chunk i is i / n of the last: the mean square of its rounding, at most 1 of it, is (i / n)^2 / 3;
        # the chunks' sums, 32 products each, add at most 32 roundings of 1 / n of it each, n of them by chance
        most = n / 3 * 1 / 3 + 32 ** 2 / n
        assert float(off.square().mean()) <= most, (name, float(off.square().mean()), most)
