"""Linear attention and the norms at a block's end together as a layer uses
them, on other streams, in captured graphs, and what the binding refuses."""
import pytest
import torch

import block_reference as bref
import gated_delta_rule_105_amd as kda
import layer_reference as ref
from gpu_util import f64, note, rel_err

pytestmark = pytest.mark.gpu


def randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


class Block:
    """Residual sum and norm, projection, convolution, norm of queries and keys, linear attention, gated norm,
    projection, residual sum and norm: H heads of d channels that share Hq queries and keys, model width D."""

    def __init__(self, D, Hq, H, d, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        self.D, self.Hq, self.H, self.d, self.dtype = D, Hq, H, d, dtype
        self.widths = [Hq * d, Hq * d, H * d, H * d, H]
        p = lambda *s: randn(g, *s)  # noqa: E731
        self.p = dict(w1=1 + 0.1 * p(D), inp=(p(D, sum(self.widths)) / D ** 0.5).to(dtype), conv=p(sum(self.widths[:3]), 4) / 2,
                      wq=1 + 0.1 * p(d), wk=1 + 0.1 * p(d), wo=1 + 0.1 * p(d), out=(p(H * d, D) / (H * d) ** 0.5).to(dtype),
                      c=0.5 + 0.1 * p(D), w2=1 + 0.1 * p(D))

    def cut(self, x, widths):
        return [t.unflatten(-1, (-1, self.d)) for t in x.split(widths, -1)]

    def forward(self, x, res, cu=None):
        p, n = self.p, sum(self.widths[:3])
        y, total = kda.residual_norm(x, res, p["w1"])
        z = y @ p["inp"]
        a, conv = kda.short_conv(z[..., :n], p["conv"], cu_seqlens=cu)
        q, k, v = self.cut(a, self.widths[:3])
        q, k = kda.qk_norm(q, k, p["wq"], p["wk"])
        g = -torch.nn.functional.softplus(z[..., -self.H:].float()).to(self.dtype)
        o, state = kda.linear_attn(q, k, v, g, cu_seqlens=cu)
        o = kda.gated_norm(o, z[..., n: n + self.H * self.d].unflatten(-1, (self.H, self.d)), p["wo"])
        return *kda.residual_norm(o.flatten(-2) @ p["out"], total, p["w2"], channel_scale=p["c"]), conv, state

    def token(self, x, res, conv, state):
        p, n = self.p, sum(self.widths[:3])
        y, total = kda.residual_norm_forward(x, res, p["w1"])
        z = y @ p["inp"]
        a = kda.short_conv_step(z[..., :n], p["conv"], conv)
        q, k, v = self.cut(a, self.widths[:3])
        q, k = kda.qk_norm_forward(q, k, p["wq"], p["wk"])
        g = -torch.nn.functional.softplus(z[..., -self.H:].float()).to(self.dtype)
        o = kda.linear_attn_step(q, k, v, state, g)
        o = kda.gated_norm_forward(o, z[..., n: n + self.H * self.d].unflatten(-1, (self.H, self.d)), p["wo"])
        return kda.residual_norm_forward(o.flatten(-2) @ p["out"], total, p["w2"], channel_scale=p["c"])

    def plain(self, x, res, cu=None):
        """The same in 64 bits; what the gradient needs."""
        p, n = {k: f64_(v) for k, v in self.p.items()}, sum(self.widths[:3])
        y, total, _, _ = bref.residual(x, res, p["w1"])
        z = y @ p["inp"]
        a, _, _ = ref.conv(z[..., :n], p["conv"], cu=cu)
        q, k, v = self.cut(a, self.widths[:3])
        qn, kn = ref.norm(q, p["wq"])[0], ref.norm(k, p["wk"])[0]
        zg = z[..., -self.H:]
        g = -torch.nn.functional.softplus(zg)
        o, ht, _, _ = bref.linear(qn, kn, v, g, cu=cu)
        gate = z[..., n: n + self.H * self.d].unflatten(-1, (self.H, self.d))
        og, _ = bref.gated(o, gate, p["wo"])
        x2 = og.flatten(-2) @ p["out"]
        y2, total2, _, _ = bref.residual(x2, total, p["w2"], p["c"])
        return dict(p=p, y=y, total=total, z=z, a=a, q=q, k=k, v=v, qn=qn, kn=kn, g=g, zg=zg, o=o, gate=gate, og=og,
                    x2=x2, y2=y2, total2=total2, ht=ht, n=n)

    def plain_grad(self, r, x, res, dy, dtotal, cu=None):
        """Gradients of <dy, y2> + <dtotal, total2>, the 64-bit forms of each part in turn."""
        p, n = r["p"], r["n"]
        e, _ = bref.residual_grad(r["x2"], r["total2"], dy, dtotal, p["w2"], p["c"])
        og = r["og"].flatten(-2)
        dog = (e["dx"] @ p["out"].T).view(r["og"].shape)
        gg, _ = bref.gated_grad(r["o"], r["gate"], dog, p["wo"])
        lg, _ = bref.linear_grad(r["qn"], r["kn"], r["v"], gg["dx"], r["g"], cu=cu)
        dq, dwq, _, _ = ref.norm_grad(r["q"], lg["dq"], p["wq"])
        dk, dwk, _, _ = ref.norm_grad(r["k"], lg["dk"], p["wk"])
        da = torch.cat([t.flatten(-2) for t in (dq, dk, lg["dv"])], -1)
        cg, _ = ref.conv_grad(r["z"][..., :n], p["conv"], da, cu=cu)
        dz = torch.cat([cg["dx"], gg["dgate"].flatten(-2), -lg["dg"] * torch.sigmoid(r["zg"])], -1)
        b, _ = bref.residual_grad(x, r["total"], dz @ p["inp"].T, e["dresidual"], p["w1"])
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        return dict(x=b["dx"], res=b["dresidual"], w1=b["dweight"], inp=flat(r["y"]).T @ flat(dz), conv=cg["dweight"],
                    wq=dwq, wk=dwk, wo=gg["dweight"], out=flat(og).T @ flat(e["dx"]), c=e["dchannel_scale"],
                    w2=e["dweight"])


def f64_(t):
    return t.detach().cpu().double()


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 4e-2)])
def test_block_prompt_and_tokens(dtype, tol):
    """A prompt and the tokens after it against the whole in 64 bits.  In bf16 ten results are rounded one after the
    other (2^-8 each at most), of inputs of one size."""
    block = Block(96, 2, 4, 32, dtype, 1)
    g = torch.Generator().manual_seed(2)
    x, res = (randn(g, 2, 105, 96, dtype=dtype) for _ in "xr")
    note(f"block {dtype}")
    T = 100
    y, total, conv, state = block.forward(x[:, :T].contiguous(), res[:, :T].contiguous())
    ys, totals = [y], [total]
    for t in range(T, 105):
        y, total = block.token(x[:, t], res[:, t], conv, state)
        ys.append(y[:, None])
        totals.append(total[:, None])
    torch.cuda.synchronize()
    r = block.plain(x, res)
    assert rel_err(f64(torch.cat(ys, 1)), r["y2"]) <= tol
    assert rel_err(f64(torch.cat(totals, 1)), r["total2"]) <= tol
    assert rel_err(f64(state), r["ht"]) <= tol


def test_block_gradients():
    """The gradients of every input and parameter through the whole block, packed sequences, against the chain of the
    64-bit forms; each part alone is held to 1e-4 of the largest element, six follow one another."""
    block = Block(96, 2, 4, 32, torch.float32, 3)
    g = torch.Generator().manual_seed(4)
    x, res, dy, dt = (randn(g, 1, 150, 96) for _ in "xryt")
    cu = torch.tensor([0, 70, 71, 150], dtype=torch.int32)
    leaves = dict(block.p, x=x, res=res)
    for t in leaves.values():
        t.requires_grad_()
    note("block gradients")
    y, total, _, _ = block.forward(x, res, cu.cuda())
    torch.autograd.backward([y, total], [dy, dt])
    torch.cuda.synchronize()
    r = block.plain(x, res, cu)
    assert rel_err(f64(y), r["y2"]) <= 1e-4
    want = block.plain_grad(r, x, res, dy, dt, cu)
    for name, w in want.items():
        assert rel_err(f64(leaves[name].grad), w) <= 6e-4, name


# ---------------------------------------------------------------- streams and graphs
def calls(seed, S=3, T=200, H=4, d=64):
    """Every entry point on inputs of its own: name -> (function of no arguments, its input tensors)."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, dtype=torch.bfloat16: randn(gen, *s, dtype=dtype)  # noqa: E731
    q, k = r(S, T, 2, d), r(S, T, 2, d)
    v, do = r(S, T, H, d), r(S, T, H, d)
    g = -r(S, T, H).abs()
    h0, w = r(S, H, d, d, dtype=torch.float32), r(d, dtype=torch.float32)
    wide, c = r(H * d, dtype=torch.float32), r(H * d, dtype=torch.float32)
    cu = torch.tensor([0, 150, 150, 431, S * T], dtype=torch.int32).cuda()
    pack = lambda t: t.reshape(1, S * T, *t.shape[2:])  # noqa: E731
    flat = lambda t: t.flatten(-2)  # noqa: E731
    return {
        "linear": (lambda: kda.linear_attn_forward(q, k, v, g, h0=h0), [q, k, v, g, h0]),
        "linear packed": (lambda: kda.linear_attn_forward(pack(q), pack(k), pack(v), pack(g), cu_seqlens=cu,
                                                          validate_cu=False), [q, k, v, g]),
        "linear grad": (lambda: kda.linear_attn_backward(q, k, v, do, g, h0=h0, dht=h0.clone()), [q, k, v, do, g, h0]),
        "linear grad packed": (lambda: kda.linear_attn_backward(pack(q), pack(k), pack(v), pack(do), pack(g),
                                                                cu_seqlens=cu, validate_cu=False), [q, k, v, do, g]),
        "gated": (lambda: kda.gated_norm_forward(v, do, w), [v, do, w]),
        "gated grad": (lambda: kda.gated_norm_backward(v, do, v.clone(), w), [v, do, w]),
        "residual": (lambda: kda.residual_norm_forward(flat(v), flat(do), wide, channel_scale=c), [v, do, wide, c]),
        "residual grad": (lambda: kda.residual_norm_backward(flat(v), flat(do), flat(v).clone(), flat(do).clone(), wide,
                                                             channel_scale=c), [v, do, wide, c]),
    }


def flat(out):
    if isinstance(out, dict):
        out = [out[k] for k in sorted(out)]
    return [t for t in (out if isinstance(out, (list, tuple)) else [out]) if t is not None]


NAMES = ["linear", "linear packed", "linear grad", "linear grad packed", "gated", "gated grad", "residual",
         "residual grad"]


@pytest.mark.parametrize("name", NAMES)
def test_other_stream(name):
    """On another current stream, with inputs made there, the same results as on the default stream."""
    note(f"stream {name}")
    fn, ins = calls(10)[name]
    want = [t.clone() for t in flat(fn())]
    side = torch.cuda.Stream()
    kept = [t.clone() for t in ins]
    for t in ins:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for t, k in zip(ins, kept):
            t.copy_(k)
        got = flat(fn())
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_explicit_stream_and_two_calls_at_once(name):
    """The same call on two streams side by side, workspaces of their own."""
    note(f"two streams {name}")
    fn, _ = calls(11)[name]
    want = [t.clone() for t in flat(fn())]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(flat(fn()))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name):
    """A captured call gives the eager call's results on every replay, with inputs changed and eager work between."""
    note(f"graph {name}")
    fn, ins = calls(12)[name]
    fn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flat(fn())
    first = [t.clone() for t in ins]
    for factor in (1.0, 0.5, 0.75):
        for t, f in zip(ins, first):
            t.copy_(f * factor)
        graph.replay()
        torch.cuda.synchronize()
        want = flat(fn())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), factor


def test_two_graphs_that_share_a_workspace():
    """Two captured forwards replayed one after the other on one stream with the same workspace."""
    note("graphs sharing a workspace")
    gen = torch.Generator().manual_seed(13)
    a = [randn(gen, 1, 900, 2, 64, dtype=torch.bfloat16) for _ in range(3)]
    b = [randn(gen, 1, 500, 2, 64, dtype=torch.bfloat16) for _ in range(3)]
    decay = torch.tensor([-0.01, -0.3], device="cuda")
    want = [kda.linear_attn_forward(*x, decay=decay) for x in (a, b)]
    ws = torch.empty(kda.linear_attn_workspace_bytes(1, 900, 2, 64, 64, torch.bfloat16), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kda.linear_attn_forward(*x, decay=decay, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
            ws.fill_(255)


def test_offsets_that_change_between_replays():
    """A captured packed call reads its offsets anew on every replay."""
    note("graph with offsets")
    gen = torch.Generator().manual_seed(14)
    q, k, v, do = (randn(gen, 1, 600, 2, 64, dtype=torch.float32) for _ in range(4))
    g = -randn(gen, 1, 600, 2).abs()
    cu = torch.tensor([0, 100, 600], dtype=torch.int32).cuda()

    def fn():
        o, ht = kda.linear_attn_forward(q, k, v, g, cu_seqlens=cu, validate_cu=False)
        return [o, ht] + flat(kda.linear_attn_backward(q, k, v, do, g, cu_seqlens=cu, validate_cu=False))
    fn()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    for offsets in ([0, 100, 600], [0, 0, 600], [0, 599, 600], [0, 320, 600]):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = fn()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), offsets


def test_explicit_stream_argument():
    note("explicit stream")
    gen = torch.Generator().manual_seed(15)
    q, k, v = (randn(gen, 1, 300, 2, 64, dtype=torch.bfloat16) for _ in range(3))
    want = kda.linear_attn_forward(q, k, v)
    y = kda.gated_norm_forward(q, k)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kda.linear_attn_forward(q, k, v, stream=s.cuda_stream)
    y2 = kda.gated_norm_forward(q, k, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(y, y2)


def test_states_updated_in_place_count_for_autograd():
    """A step writes the state that a differentiable call saved: backward through it is an error, not a wrong gradient."""
    note("state in place")
    gen = torch.Generator().manual_seed(16)
    q, k, v = (randn(gen, 2, 8, 1, 16) for _ in range(3))
    h0 = randn(gen, 2, 1, 16, 16)
    q.requires_grad_()
    o, _ = kda.linear_attn(q, k, v, h0=h0)
    kda.linear_attn_step(q.detach()[:, 0], k[:, 0], v[:, 0], h0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


# ---------------------------------------------------------------- refusals
def test_refusals():
    note("block refusals")
    x = torch.zeros(2, 8, 2, 16, device="cuda")
    g = torch.zeros(2, 8, 2, device="cuda")
    bad = [
        (lambda: kda.linear_attn_forward(x, x, x[:, :, :1]), "multiple"),
        (lambda: kda.linear_attn_forward(x, x[:, :4], x), "shape"),
        (lambda: kda.linear_attn_forward(x, x, x, g, decay=g[0, 0]), "either"),
        (lambda: kda.linear_attn_forward(x, x, x, g[:, :, :1]), "shape"),
        (lambda: kda.linear_attn_forward(x, x, x, decay=g), "shape"),
        (lambda: kda.linear_attn_forward(x, x, x, h0=torch.zeros(2, 2, 16, 15, device="cuda")), "shape"),
        (lambda: kda.linear_attn_forward(x[0], x[0], x[0]), "dimensional"),
        (lambda: kda.linear_attn_forward(x, x, x, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda")), "B == 1"),
        (lambda: kda.linear_attn_forward(x.transpose(1, 2), x.transpose(1, 2), x.transpose(1, 2)), "contiguous"),
        (lambda: kda.linear_attn_forward(x, x.cpu(), x), "cuda"),
        (lambda: kda.linear_attn_step(x[0], x[0], x[0], torch.zeros(7, 2, 16, 16, device="cuda")), "shape"),
        (lambda: kda.linear_attn_backward(x, x, x, x[:, :, :1]), "shape"),
        (lambda: kda.gated_norm_forward(x, x[:1]), "shape"),
        (lambda: kda.gated_norm_forward(x, x, activation="relu"), "activation"),
        (lambda: kda.gated_norm_forward(x, x, torch.ones(15, device="cuda")), "shape"),
        (lambda: kda.residual_norm_forward(x, x[:, :, :1]), "shape"),
        (lambda: kda.residual_norm_forward(x, x, channel_scale=torch.ones(3, device="cuda")), "shape"),
    ]
    for fn, text in bad:
        with pytest.raises(ValueError, match=text):
            fn()
    with pytest.raises(TypeError):
        kda.linear_attn_forward(x.half(), x.half(), x.half())
    with pytest.raises(TypeError):
        kda.linear_attn_forward(x, x, x, g.bfloat16())
    with pytest.raises(TypeError):
        kda.residual_norm_forward(x, x.bfloat16())
    with pytest.raises(kda.KdaError):
        kda.linear_attn_forward(*(torch.zeros(1, 4, 1, 130, device="cuda") for _ in range(3)))
    with pytest.raises(kda.KdaError):
        kda.gated_norm_forward(torch.zeros(1, 9000, device="cuda"), torch.zeros(1, 9000, device="cuda"))
    with pytest.raises(kda.KdaError):
        kda.linear_attn_forward(x, x, x, ht=x[:1].reshape(-1)[:1].new_empty(2, 2, 16, 16), o=x)
    with pytest.raises(kda.KdaError):  # a workspace that is too small
        y = torch.zeros(1, 900, 1, 64, device="cuda")
        kda.linear_attn_forward(y, y.clone(), y.clone(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_empty_batches():
    note("block empty batches")
    x = torch.zeros(2, 0, 2, 16, device="cuda")
    h0 = torch.randn(2, 2, 16, 16, device="cuda")
    o, ht = kda.linear_attn_forward(x, x, x, h0=h0)
    assert o.shape == x.shape and torch.equal(ht, h0)
    g = kda.linear_attn_backward(x, x, x, x, h0=h0, dht=2 * h0)
    assert torch.equal(g["dh0"], 2 * h0) and g["dq"].shape == x.shape
    assert kda.linear_attn_step(x[:, :0].flatten(0, 1), x.flatten(0, 1), x.flatten(0, 1),
                                torch.zeros(0, 2, 16, 16, device="cuda")).shape == (0, 2, 16)
    w = torch.ones(16, device="cuda")
    assert kda.gated_norm_forward(x, x, w).shape == x.shape
    assert (kda.gated_norm_backward(x, x, x, w)["dweight"] == 0).all()
    assert kda.residual_norm_forward(x, x, w)[0].shape == x.shape
    g = kda.residual_norm_backward(x, x, x, x, w, channel_scale=w)
    assert (g["dweight"] == 0).all() and (g["dchannel_scale"] == 0).all()
