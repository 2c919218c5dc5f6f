"""Plain 64-bit forms of the short convolution, the selective scan and the
query/key norm, token by token on the CPU, with their gradients by the chain
rule, and for every output the sum of the magnitudes of the terms it is made
of (what a relative rounding of each term can move it by).

They share no code with the library.  The gradients are themselves checked
against central differences of the forward forms in test_layer_reference.py.
"""
from __future__ import annotations

import torch


def pieces(B, T, cu):
    """(first token, end) of every sequence among the B * T tokens."""
    if cu is not None:
        c = [int(v) for v in cu]
        return list(zip(c[:-1], c[1:]))
    return [(b * T, (b + 1) * T) for b in range(B)]


def f64(t):
    return None if t is None else t.detach().cpu().double()


def silu_grad(u):
    g = torch.sigmoid(u)
    return g * (1 + u * (1 - g))


# ---------------------------------------------------------------- short convolution
def conv(x, w, bias=None, init=None, cu=None, act="silu"):
    """y, final state, and y's magnitudes."""
    x, w, bias, init = f64(x), f64(w), f64(bias), f64(init)
    B, T, D = x.shape
    W = w.shape[1]
    seqs = pieces(B, T, cu)
    xf = x.reshape(-1, D)
    y, mag = torch.zeros_like(xf), torch.zeros_like(xf)
    fin = torch.zeros(len(seqs), W - 1, D, dtype=torch.float64)
    for i, (lo, hi) in enumerate(seqs):
        before = torch.zeros(W - 1, D, dtype=torch.float64) if init is None else init[i]
        xe = torch.cat([before, xf[lo:hi]])
        for t in range(hi - lo):
            u = torch.zeros(D, dtype=torch.float64) if bias is None else bias.clone()
            m = u.abs()
            for j in range(W):
                u = u + w[:, j] * xe[t + j]
                m = m + (w[:, j] * xe[t + j]).abs()
            y[lo + t] = u * torch.sigmoid(u) if act == "silu" else u
            mag[lo + t] = m
        fin[i] = xe[hi - lo:]
    return y.reshape(x.shape), fin, mag.reshape(x.shape)


def conv_grad(x, w, dy, bias=None, init=None, dfinal=None, cu=None, act="silu"):
    """dict of gradients, and dict of their magnitudes."""
    x, w, bias, init, dy, dfinal = (f64(t) for t in (x, w, bias, init, dy, dfinal))
    B, T, D = x.shape
    W = w.shape[1]
    seqs = pieces(B, T, cu)
    xf, dyf = x.reshape(-1, D), dy.reshape(-1, D)
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    g = dict(dx=z(B * T, D), dweight=z(D, W), dbias=z(D), dinitial=z(len(seqs), W - 1, D))
    m = {k: torch.zeros_like(v) for k, v in g.items()}
    for i, (lo, hi) in enumerate(seqs):
        before = z(W - 1, D) if init is None else init[i]
        xe = torch.cat([before, xf[lo:hi]])
        dxe, mxe = torch.zeros_like(xe), torch.zeros_like(xe)
        for t in range(hi - lo):
            u = z(D) if bias is None else bias.clone()
            for j in range(W):
                u = u + w[:, j] * xe[t + j]
            du = dyf[lo + t] * (silu_grad(u) if act == "silu" else 1)
            # the derivative's own terms do not vanish where it does
            mu = dyf[lo + t].abs() * (1 + u.abs())
            for j in range(W):
                dxe[t + j] += w[:, j] * du
                mxe[t + j] += w[:, j].abs() * mu
                g["dweight"][:, j] += du * xe[t + j]
                m["dweight"][:, j] += mu * xe[t + j].abs()
            g["dbias"] += du
            m["dbias"] += mu
        if dfinal is not None:
            dxe[hi - lo:] += dfinal[i]
            mxe[hi - lo:] += dfinal[i].abs()
        g["dinitial"][i], m["dinitial"][i] = dxe[:W - 1], mxe[:W - 1]
        g["dx"][lo:hi], m["dx"][lo:hi] = dxe[W - 1:], mxe[W - 1:]
    for d in (g, m):
        d["dx"] = d["dx"].reshape(x.shape)
    return g, m


# ---------------------------------------------------------------- selective scan
def _delta(dt, bias, softplus):
    v = dt if bias is None else dt + bias
    return v, (torch.logaddexp(v, torch.zeros_like(v)) if softplus else v)


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu=None, softplus=True):
    """o, ht, and their magnitudes."""
    r = _scan_all(x, dt, A, B, C, D, z, dt_bias, h0, cu, softplus)
    return r["o"], r["ht"], r["mo"], r["mht"]


def _scan_all(x, dt, A, B, C, D, z, dt_bias, h0, cu, softplus):
    x, dt, A, B, C, D, z, dt_bias, h0 = (f64(t) for t in (x, dt, A, B, C, D, z, dt_bias, h0))
    Bt, T, ch = x.shape
    N, G = A.shape[1], B.shape[2]
    seqs = pieces(Bt, T, cu)
    xf = x.reshape(-1, ch)
    v, delta = _delta(dt.reshape(-1, ch), dt_bias, softplus)
    Bf = B.reshape(-1, G, N).repeat_interleave(ch // G, 1)
    Cf = C.reshape(-1, G, N).repeat_interleave(ch // G, 1)
    n = Bt * T
    h = torch.zeros(n, ch, N, dtype=torch.float64)
    m, before, mbefore = torch.zeros_like(h), torch.zeros_like(h), torch.zeros_like(h)
    ht = torch.zeros(len(seqs), ch, N, dtype=torch.float64)
    mht = torch.zeros_like(ht)
    a = torch.exp(delta[..., None] * A)
    for i, (lo, hi) in enumerate(seqs):
        s = torch.zeros(ch, N, dtype=torch.float64) if h0 is None else h0[i]
        ms = s.abs()
        for t in range(lo, hi):
            before[t], mbefore[t] = s, ms
            term = (delta[t] * xf[t])[:, None] * Bf[t]
            s = a[t] * s + term
            ms = a[t] * ms + term.abs()
            h[t], m[t] = s, ms
        ht[i], mht[i] = s, ms
    skip = 0 if D is None else D * xf
    y = (h * Cf).sum(-1) + skip
    my = (m * Cf.abs()).sum(-1) + (0 if D is None else (D * xf).abs())
    zf = None if z is None else z.reshape(-1, ch)
    gate = 1 if z is None else zf * torch.sigmoid(zf)
    o, mo = y * gate, my * (1 if z is None else gate.abs())
    return dict(o=o.reshape(x.shape), ht=ht, mo=mo.reshape(x.shape), mht=mht, h=h, m=m, before=before,
                mbefore=mbefore, a=a, delta=delta, v=v, x=xf, B=Bf, C=Cf, y=y, my=my, z=zf, gate=gate, seqs=seqs)


def scan_grad(x, dt, A, B, C, do, D=None, z=None, dt_bias=None, h0=None, dht=None, cu=None, softplus=True):
    """dict of gradients, and dict of their magnitudes."""
    r = _scan_all(x, dt, A, B, C, D, z, dt_bias, h0, cu, softplus)
    A, D, dht = f64(A), f64(D), f64(dht)
    Bt, T, ch = x.shape
    N, G = A.shape[1], B.shape[2]
    dof = f64(do).reshape(-1, ch)
    dy = dof * r["gate"]
    Z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    n = Bt * T
    dx, dd, mdx, mdd = Z(n, ch), Z(n, ch), Z(n, ch), Z(n, ch)
    dA, mdA = Z(ch, N), Z(ch, N)
    dB, mdB, dC, mdC = Z(n, ch, N), Z(n, ch, N), Z(n, ch, N), Z(n, ch, N)
    dh0, mdh0 = Z(len(r["seqs"]), ch, N), Z(len(r["seqs"]), ch, N)
    for i, (lo, hi) in enumerate(r["seqs"]):
        carry = Z(ch, N) if dht is None else dht[i]
        mcarry = carry.abs()
        for t in range(hi - 1, lo - 1, -1):
            dh = carry + r["C"][t] * dy[t][:, None]
            mdh = mcarry + (r["C"][t] * dy[t][:, None]).abs()
            carry, mcarry = dh * r["a"][t], mdh * r["a"][t]
            mv, mmv = carry * r["before"][t], mcarry * r["mbefore"][t]
            sB, msB = (dh * r["B"][t]).sum(-1), (mdh * r["B"][t].abs()).sum(-1)
            dx[t], mdx[t] = r["delta"][t] * sB, r["delta"][t].abs() * msB
            dd[t] = (mv * A).sum(-1) + r["x"][t] * sB
            mdd[t] = (mmv * A.abs()).sum(-1) + r["x"][t].abs() * msB
            dA += mv * r["delta"][t][:, None]
            mdA += mmv * r["delta"][t].abs()[:, None]
            q = (r["delta"][t] * r["x"][t])[:, None]
            dB[t], mdB[t] = dh * q, mdh * q.abs()
            dC[t], mdC[t] = r["h"][t] * dy[t][:, None], r["m"][t] * dy[t].abs()[:, None]
        dh0[i], mdh0[i] = carry, mcarry
    if D is not None:
        dx += D * dy
        mdx += (D * dy).abs()
    slope = torch.sigmoid(r["v"]) if softplus else torch.ones_like(r["v"])
    ddt, mddt = dd * slope, mdd * slope
    shape = x.shape
    by = lambda t: t.reshape(n, G, ch // G, N).sum(2).reshape(B.shape)  # noqa: E731
    g = dict(dx=dx.reshape(shape), ddt=ddt.reshape(shape), dA=dA, dB=by(dB), dC=by(dC), dD=(dy * r["x"]).sum(0),
             ddt_bias=ddt.sum(0), dh0=dh0)
    m = dict(dx=mdx.reshape(shape), ddt=mddt.reshape(shape), dA=mdA, dB=by(mdB), dC=by(mdC),
             dD=(dy * r["x"]).abs().sum(0), ddt_bias=mddt.sum(0), dh0=mdh0)
    if z is not None:
        g["dz"] = (dof * r["y"] * silu_grad(r["z"])).reshape(shape)
        m["dz"] = (dof.abs() * r["my"] * (1 + r["z"].abs())).reshape(shape)
    return g, m


# ---------------------------------------------------------------- norm of queries and keys
def _turn(v, pos, freq, interleaved, back=False):
    """v [.., H, d] turned; pos [..]; with the magnitudes |a| + |b| of the turned pair.  Those, and not the two
    products, because the angle is rounded too: in fp32 half turns it is off by up to 2^-25 pi, and as a product in 64
    bits by a few 2^-53 of itself (7e-7 at 2^31), which moves a cos - b sin by that share of |a sin| + |b cos|, however
    small a cos and b sin are.  That is up to 14 of the roundings allowed."""
    if freq is None or freq.numel() == 0:
        return v, v.abs()
    R = 2 * freq.numel()
    angle = pos.double()[..., None] * freq.double()
    c, s = torch.cos(angle)[..., None, :], torch.sin(angle)[..., None, :]
    if back:
        s = -s
    even = list(range(0, R, 2)) if interleaved else list(range(R // 2))
    odd = list(range(1, R, 2)) if interleaved else list(range(R // 2, R))
    a, b = v[..., even], v[..., odd]
    out, mag = v.clone(), v.abs()
    out[..., even], out[..., odd] = a * c - b * s, a * s + b * c
    mag[..., even] = mag[..., odd] = a.abs() + b.abs()
    return out, mag


def norm(x, w=None, pos=None, freq=None, norm="l2", eps=1e-6, interleaved=False, scale=1.0):
    """One of q and k [.., H, d]: output and magnitudes."""
    x, w = f64(x), f64(w)
    pos, freq = (None, None) if pos is None else (pos.cpu(), f64(freq))
    ss = (x * x).sum(-1, keepdim=True)
    v = x / torch.sqrt((ss if norm == "l2" else ss / x.shape[-1]) + eps)
    v = v if w is None else v * w
    out, mag = _turn(v, pos, freq, interleaved)
    return out * scale, mag * abs(scale)


def norm_grad(x, dout, w=None, pos=None, freq=None, norm="l2", eps=1e-6, interleaved=False, scale=1.0):
    """dx, dw and their magnitudes."""
    x, w, dout = f64(x), f64(w), f64(dout)
    pos, freq = (None, None) if pos is None else (pos.cpu(), f64(freq))
    d = x.shape[-1]
    f = 1.0 if norm == "l2" else 1.0 / d
    r = 1 / torch.sqrt(f * (x * x).sum(-1, keepdim=True) + eps)
    g, mg = _turn(dout * scale, pos, freq, interleaved, back=True)
    hat = x * r
    gw, mgw = (g, mg) if w is None else (g * w, mg * w.abs())
    dx = r * (gw - hat * (f * (gw * hat).sum(-1, keepdim=True)))
    mdx = r * (mgw + hat.abs() * (f * (mgw * hat.abs()).sum(-1, keepdim=True)))
    lead = tuple(range(x.dim() - 1))
    return dx, (g * hat).sum(lead), mdx, (mg * hat.abs()).sum(lead)


# ---------------------------------------------------------------- comparison
def check(name, got, ref, mag, roundings):
    """|got - ref| <= half a step of got's type (relative to the value) plus
    `roundings` roundings of fp32 (2^-24 each) of the magnitudes it is summed
    from, for every element."""
    assert got is not None and tuple(got.shape) == tuple(ref.shape), (name, None if got is None else got.shape)
    half = torch.finfo(got.dtype).eps / 2
    g = got.detach().cpu().double()
    room = half * ref.abs() * 1.001 + roundings * 2.0 ** -24 * mag + 1e-37
    bad = ~((g - ref).abs() <= room)
    if bad.any():
        worst = ((g - ref).abs() / room).nan_to_num(nan=float("inf"))
        at = int(worst.argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements off, the worst at {at}: got "
                             f"{g.reshape(-1)[at]:.9g}, expected {ref.reshape(-1)[at]:.9g}, allowed "
                             f"{room.reshape(-1)[at]:.3g}")
