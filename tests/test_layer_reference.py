"""The plain 64-bit forms that the layer operators are tested against: their
gradients against central differences of their forward forms."""
import pytest
import torch

import layer_reference as ref

STEP = 1e-5
# central differences in 64 bits: step^2 times a third derivative of order 10 ...
TOL = 1e-7
# ... and the rounding of f itself: a sum of a few hundred terms is off by some 64 half steps (2^-53 each) of its
# value, which the division by the step makes larger (decays above 1, which delta < 0 gives, make f large)
ROUNDINGS = 64 * 2.0 ** -53 / STEP


def directional(f, inputs, grads, seed):
    gen = torch.Generator().manual_seed(seed)
    for key, g in grads.items():
        if inputs[key] is None or g is None:
            continue
        d = torch.randn(inputs[key].shape, generator=gen, dtype=torch.float64)
        up, down = dict(inputs), dict(inputs)
        up[key], down[key] = inputs[key] + STEP * d, inputs[key] - STEP * d
        fu, fd = f(up), f(down)
        diff = (fu - fd) / (2 * STEP)
        room = TOL * (1 + abs(diff)) + ROUNDINGS * max(abs(fu), abs(fd))
        assert abs(diff - (g * d).sum()) <= room, (key, float(diff), float((g * d).sum()), float(room))


def rand(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float64)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradients(act, W):
    gen = torch.Generator().manual_seed(W)
    cu = [0, 1, 1, 9, 11]
    D, S = 3, 4
    p = dict(x=rand(gen, 1, 11, D), w=rand(gen, D, W), bias=rand(gen, D), init=rand(gen, S, W - 1, D))
    dy, dfin = rand(gen, 1, 11, D), rand(gen, S, W - 1, D)

    def f(p):
        y, fin, _ = ref.conv(p["x"], p["w"], p["bias"], p["init"], cu, act)
        return (dy * y).sum() + (dfin * fin).sum()
    g, _ = ref.conv_grad(p["x"], p["w"], dy, p["bias"], p["init"], dfin, cu, act)
    directional(f, p, dict(x=g["dx"], w=g["dweight"], bias=g["dbias"], init=g["dinitial"]), 1)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_scan_gradients(softplus, gated):
    gen = torch.Generator().manual_seed(3)
    cu, T, D, N, G = [0, 4, 4, 5, 12], 12, 4, 3, 2
    S = len(cu) - 1
    dt = rand(gen, 1, T, D)
    p = dict(x=rand(gen, 1, T, D), dt=dt if softplus else dt.abs(), A=-rand(gen, D, N).abs(), B=rand(gen, 1, T, G, N),
             C=rand(gen, 1, T, G, N), D=rand(gen, D), z=rand(gen, 1, T, D) if gated else None, dt_bias=rand(gen, D),
             h0=rand(gen, S, D, N))
    do, dht = rand(gen, 1, T, D), rand(gen, S, D, N)

    def f(p):
        o, ht, _, _ = ref.scan(cu=cu, softplus=softplus, **p)
        return (do * o).sum() + (dht * ht).sum()
    g, _ = ref.scan_grad(do=do, dht=dht, cu=cu, softplus=softplus, **p)
    directional(f, p, {k: g.get("d" + k) for k in p}, 2)


@pytest.mark.parametrize("kind", ["l2", "rms"])
@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_gradients(kind, interleaved):
    gen = torch.Generator().manual_seed(5)
    p = dict(x=rand(gen, 3, 2, 10), w=rand(gen, 10))
    pos, freq = torch.tensor([0, 7, -2]), torch.tensor([1.0, 0.3, 0.01])
    dout = rand(gen, 3, 2, 10)
    kw = dict(pos=pos, freq=freq, norm=kind, eps=0.01, interleaved=interleaved, scale=0.7)

    def f(p):
        return (dout * ref.norm(p["x"], p["w"], **kw)[0]).sum()
    dx, dw, _, _ = ref.norm_grad(p["x"], dout, p["w"], **kw)
    directional(f, p, dict(x=dx, w=dw), 4)


def test_rotation_preserves_length_and_relative_angle():
    """Turning q and k by their positions leaves q . k a function of the distance alone."""
    gen = torch.Generator().manual_seed(6)
    q, k = rand(gen, 1, 1, 8), rand(gen, 1, 1, 8)
    freq = torch.tensor([0.9, 0.2, 0.05, 0.01])
    for inter in (True, False):
        dots = []
        for base in (0, 11, 500):
            a = ref.norm(q, pos=torch.tensor([base + 3]), freq=freq, interleaved=inter)[0]
            b = ref.norm(k, pos=torch.tensor([base]), freq=freq, interleaved=inter)[0]
            assert abs(a.norm() - ref.norm(q)[0].norm()) < 1e-12
            dots.append(float((a * b).sum()))
        assert max(dots) - min(dots) < 1e-12
