"""Plain 64-bit forms of linear attention with a decay for each head (token by
token) and of the norms at a block's end, on the CPU, with their gradients by
the chain rule, and for every output the sum of the magnitudes of the terms it
is made of (what a relative rounding of each term can move it by).

They share no code with the library.  The gradients are themselves checked
against central differences of the forward forms in test_block_reference.py.
"""
from __future__ import annotations

import torch

from layer_reference import f64, pieces, silu_grad


# ---------------------------------------------------------------- linear attention
def _linear_all(q, k, v, g, decay, h0, cu, scale):
    q, k, v, g, decay, h0 = (f64(t) for t in (q, k, v, g, decay, h0))
    B, T, Hq, dk = q.shape
    H, dv = v.shape[2:]
    n = B * T
    qf, kf = (t.reshape(n, Hq, dk).repeat_interleave(H // Hq, 1) for t in (q, k))
    vf = v.reshape(n, H, dv)
    log = g.reshape(n, H) if g is not None else decay.expand(n, H) if decay is not None else torch.zeros(n, H).double()
    a = torch.exp(torch.where(log > 0, torch.zeros_like(log), log))
    seqs = pieces(B, T, cu)
    o, mo = torch.zeros_like(vf), torch.zeros_like(vf)
    S, M = torch.zeros(n, H, dk, dv).double(), torch.zeros(n, H, dk, dv).double()
    before, mbefore = torch.zeros_like(S), torch.zeros_like(S)
    ht = torch.zeros(len(seqs), H, dk, dv).double()
    mht = torch.zeros_like(ht)
    for i, (lo, hi) in enumerate(seqs):
        s = torch.zeros(H, dk, dv).double() if h0 is None else h0[i]
        m = s.abs()
        for t in range(lo, hi):
            before[t], mbefore[t] = s, m
            put = kf[t][:, :, None] * vf[t][:, None, :]
            s, m = a[t][:, None, None] * s + put, a[t][:, None, None] * m + put.abs()
            S[t], M[t] = s, m
            o[t] = scale * (qf[t][:, :, None] * s).sum(1)
            mo[t] = abs(scale) * (qf[t].abs()[:, :, None] * m).sum(1)
        ht[i], mht[i] = s, m
    return dict(q=qf, k=kf, v=vf, a=a, log=log, S=S, M=M, before=before, mbefore=mbefore, o=o.view(v.shape),
                mo=mo.view(v.shape), ht=ht, mht=mht, seqs=seqs)


def linear(q, k, v, g=None, decay=None, h0=None, cu=None, scale=1.0):
    """o, ht, and their magnitudes."""
    r = _linear_all(q, k, v, g, decay, h0, cu, scale)
    return r["o"], r["ht"], r["mo"], r["mht"]


def linear_grad(q, k, v, do, g=None, decay=None, h0=None, dht=None, cu=None, scale=1.0):
    """dict of gradients (dg also without g: by token and head), and dict of their magnitudes."""
    r = _linear_all(q, k, v, g, decay, h0, cu, scale)
    dht = f64(dht)
    dof = scale * f64(do).reshape(r["v"].shape)
    n, H, dk = r["q"].shape
    z = torch.zeros_like
    dq, dkk, dv, dlog = z(r["q"]), z(r["k"]), z(r["v"]), z(r["log"])
    mq, mk, mv, ml = z(dq), z(dkk), z(dv), z(dlog)
    dh0, mh0 = z(r["ht"]), z(r["ht"])
    for i, (lo, hi) in enumerate(r["seqs"]):
        c = z(r["ht"][i]) if dht is None else dht[i]
        mc = c.abs()
        for t in range(hi - 1, lo - 1, -1):
            ex = lambda x, y: x[:, :, None] * y[:, None, :]  # noqa: E731
            d, md = c + ex(r["q"][t], dof[t]), mc + ex(r["q"][t], dof[t]).abs()
            dq[t], mq[t] = (r["S"][t] * dof[t][:, None, :]).sum(2), (r["M"][t] * dof[t].abs()[:, None, :]).sum(2)
            dkk[t], mk[t] = (d * r["v"][t][:, None, :]).sum(2), (md * r["v"][t].abs()[:, None, :]).sum(2)
            dv[t], mv[t] = (d * r["k"][t][:, :, None]).sum(1), (md * r["k"][t].abs()[:, :, None]).sum(1)
            a = r["a"][t][:, None, None]
            c, mc = a * d, a * md
            dlog[t], ml[t] = (c * r["before"][t]).sum((1, 2)), (mc * r["mbefore"][t]).sum((1, 2))
        dh0[i], mh0[i] = c, mc
    dlog = torch.where(r["log"] > 0, z(dlog), dlog)
    share = lambda x: x.view(n, q.shape[2], H // q.shape[2], dk).sum(2).view(q.shape)  # noqa: E731
    rows = (*q.shape[:2], H)
    gr = dict(dq=share(dq), dk=share(dkk), dv=dv.view(v.shape), dg=dlog.view(rows), dh0=dh0)
    m = dict(dq=share(mq), dk=share(mk), dv=mv.view(v.shape), dg=ml.view(rows), dh0=mh0)
    return gr, m


def suffix_magnitudes(q, k, v, do, g=None, decay=None, h0=None, dht=None, cu=None, scale=1.0):
    """What dg's parts are made of when they are summed up from the end of the sequence: for every token, <|S|, |dS|> at
    its sequence's end and, of the token and those after it, |q| |dq| and |k| |dk|."""
    _, m = linear_grad(q, k, v, do, g, decay, h0, dht, cu, scale)
    r = _linear_all(q, k, v, g, decay, h0, cu, scale)
    n, H, _ = r["q"].shape
    share = H // q.shape[2]
    each = [(x.reshape(n, q.shape[2], q.shape[3]).repeat_interleave(share, 1) * y.abs()).sum(-1)
            for x, y in ((m["dq"], r["q"]), (m["dk"], r["k"]))]
    part = each[0] + each[1]
    out = torch.zeros(n, H).double()
    for i, (lo, hi) in enumerate(r["seqs"]):
        end = 0.0 if dht is None else (r["mht"][i] * f64(dht)[i].abs()).sum((1, 2))
        out[lo:hi] = part[lo:hi].flip(0).cumsum(0).flip(0) + end
    return out.view(*q.shape[:2], H)


# ---------------------------------------------------------------- norms at a block's end
def _gate(z, act):
    s = torch.sigmoid(z)
    return (z * s, silu_grad(z)) if act == "silu" else (s, s * torch.sigmoid(-z))


def gated(x, z, w=None, act="sigmoid", eps=1e-6):
    """y and its magnitudes."""
    x, z, w = f64(x), f64(z), f64(w)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = n * _gate(z, act)[0] * (1 if w is None else w)
    return y, y.abs() * (1 + z.abs())


def gated_grad(x, z, dy, w=None, act="sigmoid", eps=1e-6):
    """dict of gradients, and dict of their magnitudes."""
    x, z, w, dy = f64(x), f64(z), f64(w), f64(dy)
    w = torch.ones(x.shape[-1]).double() if w is None else w
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, (a, slope) = x * r, _gate(z, act)
    far = 1 + z.abs()  # an exponential of z is off by |z| roundings
    dn, mn = dy * w * a, (dy * w * a).abs() * far
    dx = r * (dn - n * (n * dn).mean(-1, keepdim=True))
    mx = r * (mn + n.abs() * (n.abs() * mn).mean(-1, keepdim=True))
    lead = tuple(range(x.dim() - 1))
    # the slope of SiLU is itself a sum
    ms = (torch.sigmoid(z) * (1 + (z * torch.sigmoid(-z)).abs()) if act == "silu" else slope) * far
    return (dict(dx=dx, dgate=dy * n * w * slope, dweight=(dy * n * a).sum(lead)),
            dict(dx=mx, dgate=(dy * n * w).abs() * ms, dweight=((dy * n * a).abs() * far).sum(lead)))


def residual(x, res, w=None, c=None, scale=1.0, eps=1e-6):
    """y, total, and their magnitudes."""
    x, res, w, c = f64(x), f64(res), f64(w), f64(c)
    x = scale * x * (1 if c is None else c)
    total, mag = res + x, res.abs() + x.abs()
    r = 1 / torch.sqrt((total * total).mean(-1, keepdim=True) + eps)
    by = r * (1 if w is None else w.abs())
    # the norm's statistic is off by a share of what the sum's own roundings are of it
    drift = (total.abs() * mag).mean(-1, keepdim=True) * r * r
    return total * r * (1 if w is None else w), total, by * (mag + total.abs() * (1 + drift)), mag


def residual_grad(x, total, dy, dtotal=None, w=None, c=None, scale=1.0, eps=1e-6):
    """dict of gradients, and dict of their magnitudes."""
    x, total, dy, dtotal, w, c = (f64(t) for t in (x, total, dy, dtotal, w, c))
    dn = dy if w is None else dy * w
    r = 1 / torch.sqrt((total * total).mean(-1, keepdim=True) + eps)
    n = total * r
    d = r * (dn - n * (n * dn).mean(-1, keepdim=True))
    m = r * (dn.abs() + n.abs() * (n * dn).abs().mean(-1, keepdim=True))
    if dtotal is not None:
        d, m = d + dtotal, m + dtotal.abs()
    by = scale * (1.0 if c is None else c)
    lead = tuple(range(total.dim() - 1))
    g = dict(dx=d * by, dresidual=d, dweight=(dy * n).sum(lead))
    mag = dict(dx=m * abs(by), dresidual=m, dweight=(dy * n).abs().sum(lead))
    if x is not None:
        g["dchannel_scale"], mag["dchannel_scale"] = (scale * d * x).sum(lead), abs(scale) * (m * x.abs()).sum(lead)
    return g, mag
