"""Linear attention with a decay for each head, and the norms at a block's
end, over the C ABI of ``libkda.so``.

    o, ht = linear_attn_forward(q, k, v, g)                # whole sequences
    o = linear_attn_step(q, k, v, state, g)                # one token, state in place
    y = gated_norm_forward(o, gate, weight)                # the heads' norm with the output gate
    y, total = residual_norm_forward(x, residual, weight)  # the residual sum and the next block's norm

Each has a ``*_backward`` with its gradients, and ``linear_attn``,
``gated_norm`` and ``residual_norm`` are the same as differentiable PyTorch
operations.

q, k, v, g, x, gate and residual may be column slices of a wider tensor (rows a
fixed distance apart); everything else must be contiguous.  Activations are
bfloat16 or float32, all of one dtype; parameters, fixed decays and states are
float32.  What layer.py says of offsets that nobody checks
(``validate_cu=False``) and of captured training steps holds here too.
"""
from __future__ import annotations

from ._lib import (KDA_ACT_SIGMOID, KDA_ACT_SILU, KDA_DECAY_HEAD, KDA_DECAY_NONE, KDA_DECAY_TOKEN, GatedNormDesc,
                   LinearDesc, ResidualNormDesc, layer_call, layer_workspace_size)
from .layer import (_code, _device, _ints, _like, _new, _On, _out, _rows, _sequences, _torch, _workspace, _written)

_GATES = {"sigmoid": KDA_ACT_SIGMOID, "silu": KDA_ACT_SILU}


# ---------------------------------------------------------------- linear attention
def _linear_inputs(q, k, v, g, decay, scale, lead):
    """Checks shared by the calls: device, dtype, the descriptor's fields past the batch, and the input addresses."""
    torch = _torch()
    dev, ty = _device(q, "q"), q.dtype
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError(f"q, k and v must be {lead + 2}-dimensional ([.., heads, d])")
    rows, (Hq, dk), (H, dv) = q.shape[:lead], q.shape[lead:], v.shape[lead:]
    if Hq == 0 or H % Hq:
        raise ValueError(f"the heads of v ({H}) must be a multiple of those of q and k ({Hq})")
    if g is not None and decay is not None:
        raise ValueError("either g (a log decay for each token and head) or decay (one for each head)")
    pq, ld_q = _rows("q", q, dev, ty, q.shape, lead)
    pk, ld_k = _rows("k", k, dev, ty, q.shape, lead)
    pv, ld_v = _rows("v", v, dev, ty, (*rows, H, dv), lead)
    kind, pg, ld_g = KDA_DECAY_NONE, None, 0
    if g is not None:
        kind = KDA_DECAY_TOKEN
        pg, ld_g = _rows("g", g, dev, ty, (*rows, H), lead)
    elif decay is not None:
        kind = KDA_DECAY_HEAD
        pg = _like("decay", decay, dev, torch.float32, (H,))

    def desc(B, T, n_seqs):
        return LinearDesc(*_ints(B, T, Hq, H, dk, dv, n_seqs), _code(ty), kind, scale, ld_q, ld_k, ld_v, ld_g)
    return dev, ty, (H, dk, dv), desc, (pq, pk, pv, pg)


def linear_attn_workspace_bytes(B: int, T: int, H: int, d_k: int, d_v: int, dtype, Hq: int = None,
                                n_seqs: int = 0) -> int:
    """Device workspace one linear_attn_forward call of this shape needs."""
    return layer_workspace_size("kda_linear_attn", LinearDesc(*_ints(B, T, Hq or H, H, d_k, d_v, n_seqs), _code(dtype),
                                                              KDA_DECAY_NONE, 1.0))


def linear_attn_forward(q, k, v, g=None, *, decay=None, h0=None, cu_seqlens=None, scale: float = 1.0, o=None, ht=None,
                        workspace=None, output_final_state: bool = True, validate_cu: bool = True, stream=None):
    """Linear attention with a decay for each head over whole sequences
    (kda_linear_attn_forward): S_t = exp(min(g_t, 0)) S_{t-1} + k_t v_t^T,
    o_t = scale S_t^T q_t.

    q, k: [B, T, Hq, d_k], v: [B, T, H, d_v] (bf16 or fp32, d_k and d_v up to
    128; H a multiple of Hq: head h reads q's and k's head h // (H // Hq)), or
    packed [1, sum of lengths, ..] with cu_seqlens (int32 [n + 1]).  g: log
    decays [B, T, H] in q's dtype; or decay: fp32 [H], the same for every
    token; or neither.  h0: fp32 [S, H, d_k, d_v] or None (zeros).  Returns
    (o [B, T, H, d_v], ht fp32 [S, H, d_k, d_v], or None when
    output_final_state is False).  ht must not be h0's memory."""
    f32 = _torch().float32
    dev, ty, dims, make, ptrs = _linear_inputs(q, k, v, g, decay, scale, 2)
    B, T = q.shape[:2]
    n_seqs, S, cu = _sequences(cu_seqlens, B, T, dev, validate_cu)
    p0 = _like("h0", h0, dev, f32, (S, *dims))
    desc = make(B, T, n_seqs)
    with _On(dev, stream) as st:
        need = layer_workspace_size("kda_linear_attn", desc)
        o, po = _new(o, q, "o", dev, v.shape)
        ph = None
        if ht is not None or output_final_state:
            ht, ph = _new(ht, q, "ht", dev, (S, *dims), f32)
        pws, ws_bytes, workspace = _workspace(workspace, need, dev) if need else (None, 0, None)
        layer_call("kda_linear_attn_forward", desc, *ptrs, p0, cu, po, ph, pws, ws_bytes, st)
    return o, ht


def linear_attn_step(q, k, v, state, g=None, *, decay=None, scale: float = 1.0, o=None, stream=None):
    """One token for each of N sequences: q, k [N, Hq, d_k], v [N, H, d_v], g
    [N, H]; state fp32 [N, H, d_k, d_v] is updated in place
    (kda_linear_attn_step).  Returns o [N, H, d_v]."""
    dev, ty, dims, make, ptrs = _linear_inputs(q, k, v, g, decay, scale, 1)
    N = q.shape[0]
    ps = _like("state", state, dev, _torch().float32, (N, *dims))
    if N == 0:
        return v.new_empty(v.shape) if o is None else o
    desc = make(N, 1, 0)
    with _On(dev, stream) as st:
        o, po = _new(o, q, "o", dev, v.shape)
        layer_call("kda_linear_attn_step", desc, *ptrs, ps, po, st)
    _written(state)
    return o


def linear_attn_backward(q, k, v, do, g=None, *, decay=None, h0=None, dht=None, cu_seqlens=None, scale: float = 1.0,
                         out=None, workspace=None, validate_cu: bool = True, stream=None) -> dict:
    """Gradients of <do, o> + <dht, ht> for linear_attn_forward with the same
    inputs (kda_linear_attn_backward): a dict with dq, dk, dv, dg in q's dtype
    and dh0 in fp32, each in its input's shape; dg is None without g (a fixed
    decay is a constant), dh0 without h0 unless `out` supplies it.  `out` may
    supply those tensors."""
    f32 = _torch().float32
    dev, ty, dims, make, ptrs = _linear_inputs(q, k, v, g, decay, scale, 2)
    B, T = q.shape[:2]
    n_seqs, S, cu = _sequences(cu_seqlens, B, T, dev, validate_cu)
    p0 = _like("h0", h0, dev, f32, (S, *dims))
    pdo = _like("do", do, dev, ty, v.shape)
    pdht = _like("dht", dht, dev, f32, (S, *dims))
    desc = make(B, T, n_seqs)
    out = dict(out or {})
    with _On(dev, stream) as st:
        need = layer_workspace_size("kda_linear_attn_backward", desc)
        pq, pk = _out(out, "dq", q.shape, ty, dev), _out(out, "dk", q.shape, ty, dev)
        pv = _out(out, "dv", v.shape, ty, dev)
        pg = ph = None
        if g is None:
            out["dg"] = None
        else:
            pg = _out(out, "dg", g.shape, ty, dev)
        if h0 is not None or out.setdefault("dh0", None) is not None:
            ph = _out(out, "dh0", (S, *dims), f32, dev)
        pws, ws_bytes, workspace = _workspace(workspace, need, dev) if need else (None, 0, None)
        layer_call("kda_linear_attn_backward", desc, *ptrs, p0, cu, pdo, pdht, pq, pk, pv, pg, ph, pws, ws_bytes, st)
    return out


# ---------------------------------------------------------------- the heads' norm with the output gate
def _gated_inputs(x, gate, weight, activation, eps):
    torch = _torch()
    dev, ty = _device(x, "x"), x.dtype
    if x.dim() < 2:
        raise ValueError("x and gate must be [.., heads, d]")
    if activation not in _GATES:
        raise ValueError(f"activation must be 'sigmoid' or 'silu', got {activation!r}")
    lead, (H, d) = x.dim() - 2, x.shape[-2:]
    px, ld_x = _rows("x", x, dev, ty, x.shape, lead)
    pz, ld_z = _rows("gate", gate, dev, ty, x.shape, lead)
    pw = _like("weight", weight, dev, torch.float32, (d,))
    tokens = 1
    for s in x.shape[:lead]:
        tokens *= s
    desc = GatedNormDesc(*_ints(tokens, H, d), _code(ty), _GATES[activation], eps, ld_x, ld_z)
    return dev, ty, desc, (px, pz, pw)


def gated_norm_forward(x, gate, weight=None, *, activation="sigmoid", eps: float = 1e-6, y=None, stream=None):
    """The norm of every head with its output gate, in one pass
    (kda_gated_norm_forward): y = x (mean x^2 + eps)^-1/2 weight act(gate).

    x, gate: [.., H, d] (bf16 or fp32; d up to 8192); weight: fp32 [d] or
    None; activation: "sigmoid" or "silu".  Returns y, contiguous."""
    dev, ty, desc, ptrs = _gated_inputs(x, gate, weight, activation, eps)
    with _On(dev, stream) as st:
        y, py = _new(y, x, "y", dev, x.shape)
        layer_call("kda_gated_norm_forward", desc, *ptrs, py, st)
    return y


def gated_norm_backward(x, gate, dy, weight=None, *, activation="sigmoid", eps: float = 1e-6, out=None, workspace=None,
                        stream=None) -> dict:
    """Gradients of <dy, y> for gated_norm_forward with the same inputs
    (kda_gated_norm_backward): a dict with dx, dgate in x's dtype and dweight
    fp32 [d] (None without the weight, unless `out` supplies the tensor)."""
    dev, ty, desc, ptrs = _gated_inputs(x, gate, weight, activation, eps)
    pdy = _like("dy", dy, dev, ty, x.shape)
    need = layer_workspace_size("kda_gated_norm_backward", desc)
    out = dict(out or {})
    with _On(dev, stream) as st:
        px, pz = _out(out, "dx", x.shape, ty, dev), _out(out, "dgate", x.shape, ty, dev)
        pw = None
        if weight is not None or out.setdefault("dweight", None) is not None:
            pw = _out(out, "dweight", (x.shape[-1],), _torch().float32, dev)
        pws, ws_bytes, workspace = _workspace(workspace, need, dev) if need else (None, 0, None)
        layer_call("kda_gated_norm_backward", desc, *ptrs, pdy, px, pz, pw, pws, ws_bytes, st)
    return out


# ---------------------------------------------------------------- the residual sum and the next block's norm
def _residual_inputs(like, x, residual, weight, channel_scale, scale, eps, name):
    torch = _torch()
    dev, ty = _device(like, name), like.dtype
    if like.dim() < 1:
        raise ValueError("x and residual must be [.., D]")
    lead, D = like.dim() - 1, like.shape[-1]
    px, ld_x = (None, 0) if x is None else _rows("x", x, dev, ty, like.shape, lead)
    pr, ld_r = _rows(name, residual, dev, ty, like.shape, lead)
    pw = _like("weight", weight, dev, torch.float32, (D,))
    pc = _like("channel_scale", channel_scale, dev, torch.float32, (D,))
    tokens = 1
    for s in like.shape[:lead]:
        tokens *= s
    desc = ResidualNormDesc(*_ints(tokens, D), _code(ty), scale, eps, ld_x, ld_r)
    return dev, ty, desc, (px, pr, pw, pc)


def residual_norm_forward(x, residual, weight=None, *, channel_scale=None, scale: float = 1.0, eps: float = 1e-6,
                          y=None, total=None, stream=None):
    """The residual sum behind a block and the norm before the next one, in
    one pass (kda_residual_norm_forward): total = residual + scale
    channel_scale x, y = total (mean total^2 + eps)^-1/2 weight.

    x (the block's output), residual: [.., D] (bf16 or fp32; D up to 8192);
    weight, channel_scale: fp32 [D] or None.  Returns (y, total), contiguous;
    y is the norm of the sum before it is rounded to total's dtype."""
    dev, ty, desc, ptrs = _residual_inputs(x, x, residual, weight, channel_scale, scale, eps, "residual")
    with _On(dev, stream) as st:
        y, py = _new(y, x, "y", dev, x.shape)
        total, pt = _new(total, x, "total", dev, x.shape)
        layer_call("kda_residual_norm_forward", desc, *ptrs, py, pt, st)
    return y, total


def residual_norm_backward(x, total, dy, dtotal=None, weight=None, *, channel_scale=None, scale: float = 1.0,
                           eps: float = 1e-6, out=None, workspace=None, stream=None) -> dict:
    """Gradients of <dy, y> + <dtotal, total> for residual_norm_forward, from
    the total that it returned (kda_residual_norm_backward): a dict with dx,
    dresidual in total's dtype and dweight, dchannel_scale fp32 [D] (None
    without the parameter, unless `out` supplies the tensor).  x is read for
    dchannel_scale only and may be None without.  Where the scale is 1 and
    there is no channel_scale, dx is dresidual, the same tensor, unless `out`
    supplies it."""
    dev, ty, desc, ptrs = _residual_inputs(total, x, total, weight, channel_scale, scale, eps, "total")
    pdy = _like("dy", dy, dev, ty, total.shape)
    pdt = _like("dtotal", dtotal, dev, ty, total.shape)
    f32, D = _torch().float32, total.shape[-1]
    need = layer_workspace_size("kda_residual_norm_backward", desc)
    out = dict(out or {})
    with _On(dev, stream) as st:
        pr = _out(out, "dresidual", total.shape, ty, dev)
        same = scale == 1.0 and channel_scale is None and out.get("dx") is None
        px = None if same else _out(out, "dx", total.shape, ty, dev)
        pw = pc = None
        if weight is not None or out.setdefault("dweight", None) is not None:
            pw = _out(out, "dweight", (D,), f32, dev)
        if channel_scale is not None or out.setdefault("dchannel_scale", None) is not None:
            pc = _out(out, "dchannel_scale", (D,), f32, dev)
            if x is None:
                raise ValueError("dchannel_scale needs x")
        pws, ws_bytes, workspace = _workspace(workspace, need, dev) if need else (None, 0, None)
        layer_call("kda_residual_norm_backward", desc, *ptrs, pdy, pdt, px, pr, pw, pc, pws, ws_bytes, st)
        if same:
            out["dx"] = out["dresidual"]
    return out


# ---------------------------------------------------------------- autograd
_FUNCTIONS = None


def _functions():
    """torch.autograd.Functions over the forward and backward calls (built on
    first use, so that importing the package does not import torch)."""
    global _FUNCTIONS
    if _FUNCTIONS is not None:
        return _FUNCTIONS
    torch = _torch()

    def cleared(cu, validated, **like):
        # rows behind offsets that nobody checked are not written: zeros for them
        return {} if cu is None or validated else {
            k: torch.zeros_like(t, memory_format=torch.contiguous_format) for k, t in like.items() if t is not None}

    def full(g, like):
        return torch.zeros_like(like, memory_format=torch.contiguous_format) if g is None else g.contiguous()

    class LinearAttn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g, decay, h0, cu_seqlens, scale, validate_cu):
            o, ht = linear_attn_forward(q, k, v, g, decay=decay, h0=h0, cu_seqlens=cu_seqlens, scale=scale,
                                        validate_cu=validate_cu, **cleared(cu_seqlens, validate_cu, o=v))
            ctx.save_for_backward(q, k, v, g, decay, h0, cu_seqlens)
            ctx.scale, ctx.validated = scale, validate_cu
            ctx.set_materialize_grads(False)
            return o, ht

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, do, dht):
            q, k, v, g, decay, h0, cu = ctx.saved_tensors
            r = linear_attn_backward(q, k, v, full(do, v), g, decay=decay, h0=h0,
                                     dht=None if dht is None else dht.contiguous(), cu_seqlens=cu, scale=ctx.scale,
                                     validate_cu=False, out=cleared(cu, ctx.validated, dq=q, dk=k, dv=v, dg=g))
            return r["dq"], r["dk"], r["dv"], r["dg"], None, r["dh0"], None, None, None

    class GatedNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate, weight, options):
            ctx.save_for_backward(x, gate, weight)
            ctx.options = options
            return gated_norm_forward(x, gate, weight, **options)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, gate, weight = ctx.saved_tensors
            r = gated_norm_backward(x, gate, dy.contiguous(), weight, **ctx.options)
            return r["dx"], r["dgate"], r["dweight"], None

    class ResidualNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight, channel_scale, options):
            y, total = residual_norm_forward(x, residual, weight, channel_scale=channel_scale, **options)
            ctx.save_for_backward(x if channel_scale is not None else None, total, weight, channel_scale)
            ctx.options = options
            ctx.set_materialize_grads(False)
            return y, total

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy, dtotal):
            x, total, weight, channel_scale = ctx.saved_tensors
            r = residual_norm_backward(x, total, full(dy, total), None if dtotal is None else dtotal.contiguous(),
                                       weight, channel_scale=channel_scale, **ctx.options)
            return r["dx"], r["dresidual"], r["dweight"], r["dchannel_scale"], None

    _FUNCTIONS = LinearAttn, GatedNorm, ResidualNorm
    return _FUNCTIONS


def linear_attn(q, k, v, g=None, *, decay=None, h0=None, cu_seqlens=None, scale: float = 1.0,
                validate_cu: bool = True):
    """linear_attn_forward as a differentiable PyTorch operation: returns
    (o, ht); its backward is linear_attn_backward.  A fixed decay is a constant."""
    if decay is not None and decay.requires_grad:
        raise ValueError("decay is a constant; a decay to be learned goes in as g, expanded over the tokens")
    return _functions()[0].apply(q, k, v, g, decay, h0, cu_seqlens, scale, validate_cu)


def gated_norm(x, gate, weight=None, *, activation="sigmoid", eps: float = 1e-6):
    """gated_norm_forward as a differentiable PyTorch operation: returns y;
    its backward is gated_norm_backward."""
    return _functions()[1].apply(x, gate, weight, dict(activation=activation, eps=eps))


def residual_norm(x, residual, weight=None, *, channel_scale=None, scale: float = 1.0, eps: float = 1e-6):
    """residual_norm_forward as a differentiable PyTorch operation: returns
    (y, total); its backward is residual_norm_backward."""
    return _functions()[2].apply(x, residual, weight, channel_scale, dict(scale=scale, eps=eps))
