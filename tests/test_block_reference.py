"""The plain 64-bit forms of block_reference.py: their gradients against
central differences of their forward forms (steps and tolerances as in
test_layer_reference.py), and the recurrence against the chunk form written
out as matrices."""
import pytest
import torch

import block_reference as ref
from test_layer_reference import directional, rand


@pytest.mark.parametrize("kind", ["token", "head", "none"])
@pytest.mark.parametrize("Hq,H", [(2, 2), (1, 3)])
def test_linear_gradients(kind, Hq, H):
    gen = torch.Generator().manual_seed(1)
    cu, T, dk, dv = [0, 5, 5, 6, 13], 13, 3, 4
    S = len(cu) - 1
    p = dict(q=rand(gen, 1, T, Hq, dk), k=rand(gen, 1, T, Hq, dk), v=rand(gen, 1, T, H, dv), h0=rand(gen, S, H, dk, dv),
             g=-rand(gen, 1, T, H).abs() - 0.01 if kind == "token" else None)
    if kind == "token":
        p["g"][0, 3] = 0.7  # counts as 0, and its gradient is 0
    decay = -rand(gen, H).abs() if kind == "head" else None
    do, dht = rand(gen, 1, T, H, dv), rand(gen, S, H, dk, dv)

    def f(p):
        o, ht, _, _ = ref.linear(**p, decay=decay, cu=cu, scale=0.6)
        return (do * o).sum() + (dht * ht).sum()
    g, _ = ref.linear_grad(**p, do=do, dht=dht, decay=decay, cu=cu, scale=0.6)
    grads = dict(q=g["dq"], k=g["dk"], v=g["dv"], h0=g["dh0"], g=g["dg"] if kind == "token" else None)
    directional(f, p, grads, 2)


def test_linear_against_matrices():
    """o = scale (Q K^T o D) V over the whole row, D the decays between two tokens."""
    gen = torch.Generator().manual_seed(3)
    q, k, v = rand(gen, 1, 20, 1, 5), rand(gen, 1, 20, 1, 5), rand(gen, 1, 20, 1, 6)
    g = -rand(gen, 1, 20, 1).abs()
    G = g[0, :, 0].cumsum(0)
    D = torch.exp(G[:, None] - G[None, :]).tril()
    want = 0.3 * ((q[0, :, 0] @ k[0, :, 0].T) * D) @ v[0, :, 0]
    o, ht, _, _ = ref.linear(q, k, v, g, scale=0.3)
    assert (o[0, :, 0] - want).abs().max() < 1e-13
    S = (k[0, :, 0] * torch.exp(G[-1] - G)[:, None]).T @ v[0, :, 0]
    assert (ht[0, 0] - S).abs().max() < 1e-13


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_gradients(act):
    gen = torch.Generator().manual_seed(4)
    p = dict(x=rand(gen, 2, 3, 5), z=3 * rand(gen, 2, 3, 5), w=rand(gen, 5))
    dy = rand(gen, 2, 3, 5)

    def f(p):
        return (dy * ref.gated(**p, act=act)[0]).sum()
    g, _ = ref.gated_grad(**p, dy=dy, act=act)
    directional(f, p, dict(x=g["dx"], z=g["dgate"], w=g["dweight"]), 5)


@pytest.mark.parametrize("channels", [True, False])
def test_residual_gradients(channels):
    gen = torch.Generator().manual_seed(6)
    p = dict(x=rand(gen, 4, 5), res=rand(gen, 4, 5), w=rand(gen, 5), c=rand(gen, 5) if channels else None)
    dy, dt = rand(gen, 4, 5), rand(gen, 4, 5)

    def f(p):
        y, total, _, _ = ref.residual(**p, scale=0.7)
        return (dy * y).sum() + (dt * total).sum()
    total = ref.residual(**p, scale=0.7)[1]
    g, _ = ref.residual_grad(p["x"], total, dy, dt, p["w"], p["c"], scale=0.7)
    directional(f, p, dict(x=g["dx"], res=g["dresidual"], w=g["dweight"], c=g["dchannel_scale"] if channels else None), 7)
