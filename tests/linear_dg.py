"""How far the gradients of linear attention, above all the decays', may be off: the bound that
test_gpu_linear_dg.py holds the kernels to, and what wrong sums would give,
which test_linear_dg_bounds.py shows that it rejects.

dg_t is the sum from the end of t's sequence down to t of x_s - y_s (x_s = q_s
. dq_s, y_s = k_s . dk_s, either without the token's product with itself),
beginning with <S, dS> of the end.  Each element of dq, dk and S is a sum of
terms, of which every one carries a few roundings and which are added one after
another.  Roundings have either sign, so n of them come to sqrt(n) of the
largest, here 2^-24 of the terms' magnitudes:
  an output adds 64 tokens' and 128 channels' products:      sqrt(192) = 14
  a term's weight: 128 products, a decay, three more:        sqrt(128) + 4 = 16
  a state has taken 8 additions every 32 tokens of its past: sqrt(T / 4)
K of them together.  Over channels, tokens and the elements of <S, dS> they are
independent again: the root of the sum of squares.  Half of a gradient's own
step is added for its rounding, and the whole is taken twice.
"""
from __future__ import annotations

import torch

import block_reference as ref

# the longest rows are slots of their own; `rows` of them are looked at
CASES = {
    "one-token": dict(B=1, T=1, Hq=1, H=1, dk=64, dv=64, dtype="bf16"),
    "odd-channels": dict(B=1, T=37, Hq=2, H=2, dk=13, dv=7, dtype="bf16"),
    "chunk-63": dict(B=1, T=63, Hq=1, H=2, dk=64, dv=64, dtype="bf16", state=False),
    "chunk-65": dict(B=1, T=65, Hq=1, H=1, dk=128, dv=64, dtype="bf16"),
    "chunk-33-f32": dict(B=1, T=33, Hq=2, H=2, dk=64, dv=128, dtype="f32", state=False),
    "wide": dict(B=1, T=200, Hq=1, H=2, dk=128, dv=128, dtype="bf16"),
    "wide-f32": dict(B=1, T=200, Hq=1, H=2, dk=128, dv=128, dtype="f32"),
    "narrow": dict(B=1, T=200, Hq=2, H=2, dk=3, dv=2, dtype="bf16"),
    "shared": dict(B=2, T=90, Hq=2, H=6, dk=64, dv=64, dtype="bf16"),
    "slots": dict(B=1, T=1100, Hq=2, H=2, dk=64, dv=64, dtype="bf16"),
    "slots-f32": dict(B=1, T=1100, Hq=2, H=2, dk=32, dv=64, dtype="f32"),
    "slots-across-rows": dict(B=3, T=257, Hq=1, H=2, dk=64, dv=64, dtype="f32"),
    "slots-dividing-rows": dict(B=2, T=256, Hq=1, H=1, dk=128, dv=128, dtype="bf16", state=False),
    "long-rows": dict(B=64, T=2000, Hq=4, H=4, dk=16, dv=16, dtype="bf16", rows=2),
    "long-rows-f32": dict(B=64, T=2000, Hq=2, H=4, dk=16, dv=16, dtype="f32", rows=2),
    "long-rows-no-state": dict(B=128, T=1500, Hq=2, H=2, dk=32, dv=8, dtype="bf16", rows=2, state=False),
    "packed": dict(B=1, T=0, Hq=2, H=4, dk=64, dv=64, dtype="bf16", lengths=[0, 1, 2, 0, 64, 17, 130, 1, 66, 0]),
    "packed-f32": dict(B=1, T=0, Hq=1, H=2, dk=40, dv=64, dtype="f32", lengths=[3, 300, 0, 0, 129, 1, 128, 64, 0]),
    "packed-slots": dict(B=1, T=0, Hq=2, H=6, dk=12, dv=16, dtype="bf16", lengths=[3000, 1, 0, 5400, 63, 64, 65]),
    "strong-decays": dict(B=1, T=300, Hq=2, H=2, dk=64, dv=64, dtype="f32", rate=60.0),
    "strong-decays-slots": dict(B=1, T=900, Hq=2, H=2, dk=64, dv=64, dtype="bf16", rate=30.0),
}


def inputs(name, make):
    """(arguments, offsets, gradients, the rows to look at) of a case; `make` makes them."""
    c = dict(CASES[name])
    rows = c.pop("rows", None)
    return (*make(**c, seed=41), rows)


def first(rows, p, u):
    """The first rows of a batch."""
    cut = lambda x: x[:rows] if torch.is_tensor(x) and x.dim() > 1 else x  # noqa: E731
    return {k: cut(x) for k, x in p.items()}, {k: cut(x) for k, x in u.items()}


def spread(p):
    """The inputs with q and k of each head by itself."""
    share = p["v"].shape[2] // p["q"].shape[2]
    return dict(p, **{n: p[n].repeat_interleave(share, 2) for n in "qk"})


def gradients(p, u, cu):
    """64-bit gradients of every head by itself and their magnitudes, and the recurrence's own."""
    e = {k: v.double().cpu() if torch.is_tensor(v) else v for k, v in spread(p).items()}
    d = {k: v.double().cpu() if v is not None else None for k, v in u.items()}
    return (*ref.linear_grad(**e, **d, cu=cu), ref._linear_all(e["q"], e["k"], e["v"], e["g"], e["decay"], e["h0"], cu,
                                                               e["scale"]), d["dht"])


def parts(p, u, cu):
    """64-bit dg by token and head; x - y of every token; <S, dS> of every sequence; the same as roundings count them
    (root of the sum of squares of the terms' magnitudes); the sequences."""
    return _parts(*gradients(p, u, cu))


def _parts(gr, m, r, dht):
    n, H, _ = r["q"].shape
    flat = lambda x: x.reshape(n, H, -1)  # noqa: E731
    x = (flat(gr["dq"]) * r["q"]).sum(-1) - (flat(gr["dk"]) * r["k"]).sum(-1)  # the own products cancel
    size = ((flat(m["dq"]) * r["q"]) ** 2).sum(-1) + ((flat(m["dk"]) * r["k"]) ** 2).sum(-1)
    end = torch.zeros(len(r["seqs"]), H).double() if dht is None else (r["ht"] * dht).sum((2, 3))
    end_size = torch.zeros_like(end) if dht is None else ((r["mht"] * dht) ** 2).sum((2, 3))
    return gr["dg"], x, end, size, end_size, r["seqs"]


def suffix(x, end, seqs, cut=None):
    """Sums from the end of each sequence; `cut`: they begin anew, from nothing, at its multiples."""
    out = torch.zeros_like(x)
    for i, (lo, hi) in enumerate(seqs):
        ends = [hi] if cut is None else [b for b in range((lo // cut + 1) * cut, hi, cut)] + [hi]
        at = lo
        for b in ends:
            if b > at:
                out[at:b] = x[at:b].flip(0).cumsum(0).flip(0) + (end[i] if b == hi else 0.0)
            at = b
    return out


def bounds(p, u, cu, dtype):
    """{name: (64-bit gradient, what it may be off by)} of dg and the others."""
    gr, m, r, dht = gradients(p, u, cu)
    dg, _, _, size, end_size, seqs = _parts(gr, m, r, dht)
    longest = max((hi - lo for lo, hi in seqs), default=1)
    K = 14 + 16 + (longest / 4) ** 0.5
    noise = {"dg": suffix(size, end_size, seqs).sqrt().view(dg.shape), "dv": m["dv"], "dh0": m["dh0"]}
    shared = lambda x: x.unflatten(2, (p["q"].shape[2], -1)).sum(3)  # noqa: E731
    for k in ("dq", "dk"):
        gr[k], noise[k] = shared(gr[k]), shared(m[k])
    half = {k: 2.0 ** -24 if k == "dh0" else torch.finfo(dtype).eps / 2 for k in noise}
    return {k: (gr[k], 2 * (2.0 ** -24 * K * noise[k] + half[k] * gr[k].abs()) + 1e-37) for k in noise}
