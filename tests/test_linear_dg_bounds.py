"""The bound on linear attention's dg (linear_dg.py) rejects, in every case,
zeros, sums without <S, dS> of the sequence's end, and sums that begin anew
every 64 tokens."""
import pytest
import torch

import linear_dg
import test_gpu_linear_attn as linear


@pytest.mark.parametrize("name", linear_dg.CASES)
def test_wrong_sums_are_rejected(name, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t)
    p, cu, u, rows = linear_dg.inputs(name, linear.inputs)
    dtype = p["q"].dtype
    if rows:
        p, u = linear_dg.first(rows, p, u)
    dg, room = linear_dg.bounds(p, u, cu, dtype)["dg"]
    _, x, end, _, _, seqs = linear_dg.parts(p, u, cu)

    def rejected(sums):
        return float(((sums.view(dg.shape) - dg).abs() > room).double().mean())
    # of strong decays one head of two keeps a gradient that is not below the terms' roundings
    most = 0.5 if name.startswith("strong") else 0.9
    assert rejected(linear_dg.suffix(x, end, seqs)) == 0
    assert rejected(torch.zeros_like(dg)) > most
    if u["dht"] is not None:
        assert rejected(linear_dg.suffix(x, 0 * end, seqs)) > most
    longest = max(hi - lo for lo, hi in seqs)
    if longest > 64:
        assert rejected(linear_dg.suffix(x, end, seqs, 64)) > 0.1
    if most == 0.9:
        assert float((room / dg.abs().clamp(min=1e-30)).median()) <= (0.02 if dtype is torch.bfloat16 else 0.005)
