"""The operators around the recurrence at values where padding, composed
decays or bookkeeping could show: no epsilon, growing states, infinities next
to lanes that have no state or channel, rows behind the last sequence, states
that are updated in place while a gradient still needs them."""
import pytest
import torch

import gated_delta_rule_105_amd as kda
import layer_reference as ref
import test_gpu_qk_norm as norm_cases
from gpu_util import note
from layer_reference import check

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norm without an epsilon
@pytest.mark.parametrize("Hq,Hk,d,rot", [(3, 1, 128, 0), (5, 4, 64, 64), (3, 1, 34, 34), (5, 1, 32, 16), (1, 1, 512, 0)])
@pytest.mark.parametrize("kind", ["l2", "rms"])
def test_norm_gradient_without_epsilon(Hq, Hk, d, rot, kind):
    """eps = 0 is allowed; the lanes of a wave beyond the last head, whose norm would be zero, add nothing to the
    weights' gradients.  Roundings as in test_gpu_qk_norm."""
    p = norm_cases.inputs((2, 23), Hq, Hk, d, rot, "f32", seed=40)
    note(f"qk_norm_backward eps 0 Hq={Hq} Hk={Hk} d={d} {kind}")
    g = kda.qk_norm_backward(p["q"], p["k"], p["dq"], p["dk"], p["wq"], p["wk"], p["pos"], p["freq"], norm=kind, eps=0.0)
    torch.cuda.synchronize()
    for n, x, w, dout in (("q", p["q"], p["wq"], p["dq"]), ("k", p["k"], p["wk"], p["dk"])):
        dx, dw, mx, mw = ref.norm_grad(x, dout, w, p["pos"], p["freq"], kind, 0.0)
        check("d" + n, g["d" + n], dx, mx, 128)
        check(f"d{n}_weight", g[f"d{n}_weight"], dw, mw, 128 + x.numel() // d)


# ---------------------------------------------------------------- states that grow and shrink
def swinging(lengths, seed):
    """64-token stretches with steps of either sign: half of the states (tiny ones, with tiny B and C) grow by e^102 in
    a stretch and shrink back in the next, the others swing the other way by e^-26."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    T, D, N = 384, 10, 6
    S = 1 if lengths is None else len(lengths)
    cu = None if lengths is None else torch.tensor([sum(lengths[:i]) for i in range(S + 1)], dtype=torch.int32).cuda()
    size = torch.ones(N).cuda()
    size[::2] = 1e-20
    dt = torch.tensor([0.0, 0.8, -0.8, 0.75, -0.75, 0.1]).repeat_interleave(64).cuda()
    A = torch.full((D, N), -0.5).cuda()
    A[:, ::2] = 2.0
    p = dict(x=r(1, T, D), dt=dt[None, :, None].expand(1, T, D).contiguous(), A=A, B=r(1, T, 1, N) * size,
             C=r(1, T, 1, N) * size, D=r(D), z=r(1, T, D))
    return p, r(S, D, N) * size, cu, r(1, T, D), r(S, D, N) * size


@pytest.mark.parametrize("lengths", [None, [70, 0, 314], [1, 383]])
def test_states_that_swing(lengths):
    """Every state stays inside fp32 token by token, so composing stretches must not overflow either.  A step
    multiplies by e^1.6, off by under 7 roundings; a stretch of 64 composed at once is off by its sum of delta (16
    additions a lane and 2 more, 9 roundings at half their weight) times its exponent of 103: under 1024 roundings, 16
    a token.  The gradient has two such recurrences."""
    p, h0, cu, do, dht = swinging(lengths, 50)
    note(f"selective_scan swinging states {lengths}")
    o, ht = kda.selective_scan_forward(**p, h0=h0, cu_seqlens=cu, dt_softplus=False)
    g = kda.selective_scan_backward(**p, do=do, h0=h0, dht=dht, cu_seqlens=cu, dt_softplus=False)
    torch.cuda.synchronize()
    ro, rht, mo, mht = ref.scan(**p, h0=h0, cu=cu, softplus=False)
    check("o", o, ro, mo, 64 + 16 * 384)
    check("ht", ht, rht, mht, 64 + 16 * 384)
    rg, rm = ref.scan_grad(**p, do=do, h0=h0, dht=dht, cu=cu, softplus=False)
    for key in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dh0"):
        check(key, g[key], rg[key], rm[key], 128 + 32 * 384 + 384)


def test_a_state_that_vanishes_and_grows():
    """Stretches that decay by 2^-550 and then grow by as much leave what fp32 leaves of a state, never a NaN."""
    p, h0, _, do, dht = swinging(None, 51)
    note("selective_scan vanishing states")
    long = lambda t: t.repeat(1, 4, *[1] * (t.dim() - 2))  # noqa: E731
    p = {k: (long(v) if k in ("x", "B", "C", "z") else v) for k, v in p.items()}
    p["dt"] = torch.tensor([-3.0, 3.0] * 12).repeat_interleave(64).cuda()[None, :, None].expand(1, 1536, 10).contiguous()
    p["B"][..., ::2] = 0.0
    p["A"][:, 1::2] = -0.01
    o, ht = kda.selective_scan_forward(**p, h0=h0, dt_softplus=False)
    do = long(do)
    p["C"][..., ::2] = 0.0
    g = kda.selective_scan_backward(**p, do=do, h0=h0, dt_softplus=False)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all() and torch.isfinite(ht).all()
    for key in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dh0"):
        assert torch.isfinite(g[key]).all(), key


# ---------------------------------------------------------------- infinities beside lanes without a state or channel
def positive(D, N, dtype, seed, T=150):
    """Positive inputs and slow decays: an infinity stays one of its sign through every sum."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: 0.1 + torch.rand(*s, generator=gen)  # noqa: E731
    c = lambda *s: r(*s).to(dtype).cuda()  # noqa: E731
    p = dict(x=c(1, T, D), dt=(r(1, T, D) - 2).to(dtype).cuda(), A=(-0.01 * r(D, N)).cuda(), B=c(1, T, 1, N),
             C=c(1, T, 1, N), D=r(D).cuda(), z=c(1, T, D))
    return p, r(1, D, N).cuda(), c(1, T, D), r(1, D, N).cuda()


def same_kind(name, got, want):
    """NaN, infinities and their signs where the definition has them."""
    got, want = got.detach().cpu().double(), want
    for kind, a, b in (("nan", got.isnan(), want.isnan()), ("inf", got == float("inf"), want == float("inf")),
                       ("-inf", got == -float("inf"), want == -float("inf"))):
        assert torch.equal(a, b), f"{name}: {int((a != b).sum())} of {a.numel()} elements differ in being {kind}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,N", [(18, 1), (18, 3), (16, 4), (18, 6), (20, 12), (18, 16), (16, 17), (18, 24), (18, 33),
                                 (17, 48)])
@pytest.mark.parametrize("where", ["x", "B", "C", "h0", "dht", "do"])
def test_infinities_next_to_padding(where, D, N, dtype):
    """N and D that leave lanes without a state or a channel: an infinity gives what the definition gives."""
    p, h0, do, dht = positive(D, N, dtype, 60 + N)
    note(f"selective_scan infinity in {where} D={D} N={N} {dtype}")
    t = dict(p, h0=h0, do=do, dht=dht)[where]
    t.reshape(-1)[(70 * t[0, 0].numel() if t.dim() > 2 and t.shape[1] == 150 else 0) + t[0, 0].numel() - 1] = float("inf")
    if where in ("h0", "dht"):
        t.zero_()[0, D - 1, N - 1] = float("inf")
    o, ht = kda.selective_scan_forward(**p, h0=h0)
    g = kda.selective_scan_backward(**p, do=do, h0=h0, dht=dht)
    torch.cuda.synchronize()
    ro, rht, _, _ = ref.scan(**p, h0=h0)
    same_kind("o", o, ro)
    same_kind("ht", ht, rht)
    rg, _ = ref.scan_grad(**p, do=do, h0=h0, dht=dht)
    for key in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dh0"):
        same_kind(key, g[key], rg[key])
    state = h0.clone()
    for i in range(150):
        tok = {k: (v[:, i] if k in ("x", "dt", "z", "B", "C") else v) for k, v in p.items()}
        oi = kda.selective_scan_step(state=state, **tok)
        if 68 <= i < 74:
            same_kind(f"step {i}", oi, ro[:, i])


# ---------------------------------------------------------------- rows behind the last sequence
def soiled(*shape, dtype):
    """Leaves NaN in the memory that the next tensor of this size is made of."""
    torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_behind_the_last_sequence(dtype):
    """Offsets that nobody checks (as in a captured graph) and that end before the batch does: the differentiable
    forms give zeros there, and gradients of zero, in place of what the memory held."""
    gen = torch.Generator().manual_seed(70)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()  # noqa: E731
    T, end, D, N = 190, 131, 24, 8
    cu = torch.tensor([0, 40, end], dtype=torch.int32).cuda()
    f = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    note(f"rows behind the last sequence {dtype}")
    for _ in range(8):
        soiled(1, T, D, dtype=dtype)
        soiled(1, T, 1, N, dtype=dtype)
    x, w, dy = r(1, T, D), f(D, 4), r(1, T, D)
    lead = lambda t: t[:, :end].contiguous()  # noqa: E731
    xl = x.clone().requires_grad_()
    y, _ = kda.short_conv(xl, w, cu_seqlens=cu, validate_cu=False)
    y.backward(dy)
    ys, _ = kda.short_conv_forward(lead(x), w, cu_seqlens=cu)
    gs = kda.short_conv_backward(lead(x), w, lead(dy), cu_seqlens=cu)
    for got, want in ((y, ys), (xl.grad, gs["dx"])):
        assert torch.equal(got[:, :end], want) and not got[:, end:].any()
    p = dict(x=r(1, T, D), dt=r(1, T, D), A=-torch.exp(f(D, N)), B=r(1, T, 1, N), C=r(1, T, 1, N), D=f(D), z=r(1, T, D),
             dt_bias=f(D))
    do = r(1, T, D)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    o, _ = kda.selective_scan(**leaves, cu_seqlens=cu, validate_cu=False)
    o.backward(do)
    torch.cuda.synchronize()
    cut = {k: (lead(v) if k in ("x", "dt", "B", "C", "z") else v) for k, v in p.items()}
    ro, _, mo, _ = ref.scan(**cut, cu=cu)
    check("o", o[:, :end], ro, mo, 64 + 8 * end)
    assert not o[:, end:].any()
    rg, rm = ref.scan_grad(**cut, do=lead(do), cu=cu)
    for key in ("x", "dt", "B", "C", "z"):
        check("d" + key, leaves[key].grad[:, :end], rg["d" + key], rm["d" + key], 128 + 16 * end)
        assert not leaves[key].grad[:, end:].any(), key
    for key in ("A", "D", "dt_bias"):
        check("d" + key, leaves[key].grad, rg["d" + key], rm["d" + key], 128 + 17 * end)


def test_rows_behind_the_last_sequence_in_a_graph():
    """One captured call serves batches of other lengths: the offsets are rewritten between replays, and each replay
    gives what an eager call gives, zeros behind the last sequence among it."""
    gen = torch.Generator().manual_seed(71)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    T, D, N = 300, 40, 12
    cu = torch.tensor([0, 100, 300], dtype=torch.int32).cuda()
    x, dt, z, w = r(1, T, D), r(1, T, D), r(1, T, D), r(D, 4)
    A, B, C = -torch.exp(r(D, N)), r(1, T, 1, N), r(1, T, 1, N)
    note("rows behind the last sequence in a graph")

    def call():
        y, conv = kda.short_conv(x, w, cu_seqlens=cu, validate_cu=False)
        o, h = kda.selective_scan(y, dt, A, B, C, None, z, cu_seqlens=cu, validate_cu=False)
        return y, conv, o, h
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for ends in ([0, 100, 300], [0, 7, 90], [0, 0, 0], [0, 299, 300]):
        cu.copy_(torch.tensor(ends, dtype=torch.int32))
        x.copy_(r(1, T, D))
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), ends
        assert not out[0][:, ends[-1]:].any() and not out[2][:, ends[-1]:].any(), ends


# ---------------------------------------------------------------- states updated in place
def test_updates_in_place_are_seen_by_autograd():
    """A state that a gradient still needs and that a step then overwrites is an error, as with any operation in
    place, and not a wrong gradient; so is an output written over an input that was kept."""
    gen = torch.Generator().manual_seed(80)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    D, N, T = 8, 4, 20
    note("updates in place")
    w, x = r(D, 4).requires_grad_(), r(1, T, D)
    conv = r(1, 3, D)
    y, _ = kda.short_conv(x, w, initial_state=conv)
    kda.short_conv_step(x[:, 0], w, conv)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    A, B, C, h = (-torch.exp(r(D, N))).requires_grad_(), r(1, T, 1, N), r(1, T, 1, N), r(1, D, N)
    o, _ = kda.selective_scan(x, x, A, B, C, h0=h)
    kda.selective_scan_step(x[:, 0], x[:, 0], A, B[:, 0], C[:, 0], h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()
    q = r(2, 5, 2, 32)
    k, wq = r(2, 5, 2, 32), r(32).requires_grad_()
    out, _ = kda.qk_norm(q, k, wq)
    kda.qk_norm_forward(k, k, q_out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    out, _ = kda.qk_norm(q, k, wq)
    kda.qk_norm_backward(k, k, k, k, out=dict(dq=q))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    with torch.inference_mode():  # tensors that have no version
        conv, h = r(1, 3, D), r(1, D, N)
        y = kda.short_conv_step(x[:, 0], w, conv)
        kda.selective_scan_step(y, y, A, B[:, 0], C[:, 0], h)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- angles beside a quarter turn's multiples
def test_angles_beside_quarter_turns():
    """fp32 angles next to multiples of a quarter turn: the small one of cosine and sine keeps its relative accuracy.
    The unit vector (1, 0) gives both as they are.  The product and the turn are off by a few 2^-53 of the angle, the
    rest of the turn is rounded once (2^-24 of itself), cosine and sine take under 4 roundings each."""
    note("qk_norm quarter turns")
    gen = torch.Generator().manual_seed(90)
    quarter = torch.tensor(torch.pi / 2).float()
    freq = quarter * torch.tensor([1.0, 2.0, 3.0, 5.0, 0.25]) * (1 + torch.randint(-4, 5, (5,), generator=gen) * 2.0 ** -23)
    pos = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 100, 4099, -3, -1026], dtype=torch.int32)
    outs = []
    for i in range(5):  # one pair at a time, so that the vector is a unit
        x = torch.zeros(len(pos), 1, 10)
        x[..., i] = 1.0
        outs.append(kda.qk_norm_forward(x.cuda(), x.cuda(), None, None, pos.cuda(), freq.cuda(), eps=0.0)[0].cpu())
    angle = pos.double()[:, None] * freq.double()
    room = 8 * 2.0 ** -53 * angle.abs()
    for i in range(5):
        for at, want in ((i, torch.cos(angle[:, i])), (5 + i, torch.sin(angle[:, i]))):
            got = outs[i][:, 0, at].double()
            assert ((got - want).abs() <= 6 * 2.0 ** -24 * want.abs() + room[:, i]).all(), (i, at)
