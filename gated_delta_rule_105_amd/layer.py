"""The operators around the recurrence in a layer, over the C ABI of
``libkda.so``: the short causal convolution and the norm of queries and keys
(with the position rotation) that make a layer's q, k and v, and the selective
state space scan.

    y, state = short_conv_forward(x, weight, bias)        # whole sequences
    y = short_conv_step(x, weight, state, bias)           # one token, state in place
    q, k = qk_norm_forward(q, k, q_weight, k_weight, positions, inv_freq)
    o, ht = selective_scan_forward(x, dt, A, B, C, D, z, dt_bias)
    o = selective_scan_step(x, dt, A, B, C, state, D, z, dt_bias)

Each has a ``*_backward`` with its gradients, and ``short_conv``, ``qk_norm``
and ``selective_scan`` are the same as differentiable PyTorch operations.

x, dt, z, B, C, q and k may be column slices of a wider tensor (rows a fixed
distance apart); everything else must be contiguous.  Activations are bfloat16
or float32, all of one dtype; parameters and states of the scan are float32.

In a captured graph pass ``validate_cu=False`` (the check reads the offsets on
the host).  Offsets that then end before the batch does leave rows behind the
last sequence, which no call writes: tensors that a call makes hold there what
the memory held, tensors handed in keep what they had, and the differentiable
forms, which would hand such rows on as gradients, fill their own with zeros.
To capture a training step, call the ``*_backward`` functions: a
captured ``.backward()`` must not meet leaves whose earlier autograd graph,
made outside the capture, is still alive (PyTorch would tie the capture to
the stream of that graph).
"""
from __future__ import annotations

from ._lib import (KDA_ACT_NONE, KDA_ACT_SILU, KDA_DTYPE_BF16, KDA_DTYPE_F32, KDA_NORM_RMS, KDA_NORM_UNIT, ConvDesc,
                   NormDesc, ScanDesc, layer_call, layer_workspace_size)

_ACTIVATIONS = {"silu": KDA_ACT_SILU, "none": KDA_ACT_NONE, None: KDA_ACT_NONE}
_NORMS = {"l2": KDA_NORM_UNIT, "rms": KDA_NORM_RMS}

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _code(dtype) -> int:
    torch = _torch()
    if dtype is torch.bfloat16:
        return KDA_DTYPE_BF16
    if dtype is torch.float32:
        return KDA_DTYPE_F32
    raise TypeError(f"unsupported dtype {dtype}; the library takes bfloat16 or float32")


def _ints(*lengths):
    """`lengths`, which the descriptors hold in 32 bits (ctypes would wrap longer ones)."""
    if max(lengths) > 0x7fffffff:
        raise ValueError(f"lengths are limited to 2^31 - 1, got {max(lengths)}")
    return lengths


def _elsewhere(name, t, dev):
    return ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _like(name, t, dev, dtype, shape):
    """Check an optional contiguous tensor on device number `dev`; returns its address (None for None)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise _elsewhere(name, t, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(name, t, dev, dtype, shape, lead):
    """Check an input whose rows (the dims from `lead` on) are contiguous and a
    fixed distance apart; returns its address and that distance (0: none
    needed, the rows follow one another)."""
    if t.get_device() != dev:
        raise _elsewhere(name, t, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    size, stride = t.shape, t.stride()
    # the usual slice, [B, T, row] or [N, row] with rows of one or two dims, without the loops
    inner = len(size) - lead
    if stride[-1] == 1 and (inner == 1 or (inner == 2 and stride[-2] == size[-1])) and lead <= 2:
        row = size[-1] if inner == 1 else size[-1] * size[-2]
        ld = stride[lead - 1]
        if ld >= row and size[lead - 1] > 1 and (lead == 1 or size[0] == 1 or stride[0] == ld * size[1]):
            return t.data_ptr(), ld
    row = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if size[i] != 1 and stride[i] != row:
            raise ValueError(f"the last {t.dim() - lead} dims of {name} must be contiguous")
        row *= size[i]
    ld, tokens = 0, 1
    for i in range(lead - 1, -1, -1):
        if size[i] == 1:
            continue
        if tokens == 1:
            ld = stride[i]
            if ld < row:
                raise ValueError(f"the rows of {name} overlap")
        elif stride[i] != ld * tokens:
            raise ValueError(f"the token rows of {name} must be a fixed distance apart")
        tokens *= size[i]
    return t.data_ptr(), ld


def _device(t, name):
    """The number of the device a call's tensors have to be on."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _sequences(cu_seqlens, B, T, dev, validate_cu):
    """(number of packed sequences or 0, sequences, address of the offsets)"""
    if cu_seqlens is None:
        return 0, B, None
    torch = _torch()
    if B != 1:
        raise ValueError("packed sequences need B == 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a vector of at least two offsets")
    cu = _like("cu_seqlens", cu_seqlens, dev, torch.int32, cu_seqlens.shape)
    if validate_cu:
        from . import check_cu_seqlens
        check_cu_seqlens(cu_seqlens.cpu(), T)
    n = cu_seqlens.numel() - 1
    return n, n, cu


class _On:
    """The device and stream a call runs on: the tensors' device is made the
    current one, and with an explicit stream torch allocates from that
    stream's pool (so that a workspace freed on return is not handed to other
    work while the stream still uses it)."""

    __slots__ = ("device", "stream", "contexts")

    def __init__(self, device, stream):
        self.device = device
        self.stream = stream
        self.contexts = ()

    def __enter__(self):
        torch = _torch()
        if self.stream is not None:
            self.contexts = (torch.cuda.device(self.device),
                             torch.cuda.stream(torch.cuda.ExternalStream(self.stream, device=self.device)))
        elif torch._C._cuda_getDevice() != self.device:
            self.contexts = (torch.cuda.device(self.device),)
        for c in self.contexts:
            c.__enter__()
        # the handle alone: torch.cuda.current_stream() would build a Stream around it on every call
        return torch._C._cuda_getCurrentRawStream(self.device) if self.stream is None else self.stream

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _written(t):
    """Tell autograd that a caller's tensor is written, which it cannot see: a gradient that still needs what the
    tensor held is then an error."""
    _torch().autograd.graph.increment_version(t)


def _new(t, like, name, dev, shape, dtype=None):
    """A caller's output, checked, or a new one (in `like`'s dtype unless given); and its address."""
    if t is None:
        t = like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)
        return t, t.data_ptr()
    address = _like(name, t, dev, like.dtype if dtype is None else dtype, shape)
    _written(t)
    return t, address


def _out(out, name, shape, dtype, dev):
    """The caller's tensor under `name`, checked, or a new one; its address."""
    t = out.get(name)
    if t is None:
        t = _torch().empty(shape, dtype=dtype, device=dev)
        out[name] = t
        return t.data_ptr()
    address = _like(name, t, dev, dtype, shape)
    _written(t)
    return address


def _workspace(workspace, need, dev):
    """Address and bytes of a uint8 workspace of at least `need` bytes, and its tensor."""
    torch = _torch()
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# ---------------------------------------------------------------- short convolution
def _activation(name):
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or 'none', got {name!r}")
    return _ACTIVATIONS[name]


def _conv_desc(x, weight, B, T, D, W, n_seqs, activation, ld):
    return ConvDesc(*_ints(B, T, D, W, n_seqs), _code(x.dtype), _activation(activation), ld)


def short_conv_forward(x, weight, bias=None, *, initial_state=None, cu_seqlens=None, activation="silu", y=None,
                       final_state=None, output_final_state: bool = True, validate_cu: bool = True, stream=None):
    """Short causal convolution over whole sequences, one filter per channel
    (kda_short_conv_forward): y_t = act(bias + sum_j weight[:, j] x[t - (W - 1) + j]).

    x: [B, T, D] (bf16 or fp32), or [1, sum of lengths, D] with cu_seqlens
    (int32 [n + 1]); weight: fp32 [D, W], W in 2 .. 4; bias: fp32 [D] or None;
    activation: "silu" or "none".  initial_state: [S, W - 1, D] in x's dtype,
    the inputs before each sequence, oldest first (None: zeros).  Returns
    (y [B, T, D], final_state [S, W - 1, D], or None when output_final_state
    is False); final_state is the next call's initial_state."""
    torch = _torch()
    dev, dt = _device(x, "x"), x.dtype
    B, T, D = x.shape
    W = weight.shape[-1]
    px, ld = _rows("x", x, dev, dt, x.shape, 2)
    pw = _like("weight", weight, dev, torch.float32, (D, W))
    pb = _like("bias", bias, dev, torch.float32, (D,))
    n_seqs, S, cu = _sequences(cu_seqlens, B, T, dev, validate_cu)
    p0 = _like("initial_state", initial_state, dev, dt, (S, W - 1, D))
    desc = _conv_desc(x, weight, B, T, D, W, n_seqs, activation, ld)
    with _On(dev, stream) as st:
        y, py = _new(y, x, "y", dev, (B, T, D))
        pf = None
        if final_state is not None or output_final_state:
            final_state, pf = _new(final_state, x, "final_state", dev, (S, W - 1, D))
        layer_call("kda_short_conv_forward", desc, px, pw, pb, p0, cu, py, pf, st)
    return y, final_state


def short_conv_step(x, weight, state, bias=None, *, activation="silu", y=None, stream=None):
    """One token for each of N sequences: x [N, D]; state [N, W - 1, D] in x's
    dtype is updated in place (kda_short_conv_step).  Returns y [N, D]."""
    torch = _torch()
    dev, dt = _device(x, "x"), x.dtype
    N, D = x.shape
    W = weight.shape[-1]
    px, ld = _rows("x", x, dev, dt, x.shape, 1)
    pw = _like("weight", weight, dev, torch.float32, (D, W))
    pb = _like("bias", bias, dev, torch.float32, (D,))
    ps = _like("state", state, dev, dt, (N, W - 1, D))
    if N == 0:
        return x.new_empty((0, D)) if y is None else y
    desc = _conv_desc(x, weight, N, 1, D, W, 0, activation, ld)
    with _On(dev, stream) as st:
        y, py = _new(y, x, "y", dev, (N, D))
        layer_call("kda_short_conv_step", desc, px, pw, pb, ps, py, st)
    _written(state)
    return y


def short_conv_backward(x, weight, dy, bias=None, *, initial_state=None, dfinal=None, cu_seqlens=None,
                        activation="silu", out=None, workspace=None, validate_cu: bool = True, stream=None) -> dict:
    """Gradients of <dy, y> + <dfinal, final_state> for short_conv_forward
    with the same inputs (kda_short_conv_backward): a dict with dx [B, T, D]
    and dinitial [S, W - 1, D] in x's dtype, dweight fp32 [D, W] and dbias
    fp32 [D]; dbias and dinitial are None without a bias or an initial state.
    `out` may supply those tensors; given there, they are written either way."""
    torch = _torch()
    dev, dt, f32 = _device(x, "x"), x.dtype, torch.float32
    B, T, D = x.shape
    W = weight.shape[-1]
    px, ld = _rows("x", x, dev, dt, x.shape, 2)
    pw = _like("weight", weight, dev, f32, (D, W))
    pb = _like("bias", bias, dev, f32, (D,))
    n_seqs, S, cu = _sequences(cu_seqlens, B, T, dev, validate_cu)
    p0 = _like("initial_state", initial_state, dev, dt, (S, W - 1, D))
    pdy = _like("dy", dy, dev, dt, (B, T, D))
    pdf = _like("dfinal", dfinal, dev, dt, (S, W - 1, D))
    desc = _conv_desc(x, weight, B, T, D, W, n_seqs, activation, ld)
    need = layer_workspace_size("kda_short_conv_backward", desc)
    out = dict(out or {})
    with _On(dev, stream) as st:
        pdx = _out(out, "dx", (B, T, D), dt, dev)
        pdw = _out(out, "dweight", (D, W), f32, dev)
        pdb = pdi = None
        if bias is not None or out.setdefault("dbias", None) is not None:
            pdb = _out(out, "dbias", (D,), f32, dev)
        if initial_state is not None or out.setdefault("dinitial", None) is not None:
            pdi = _out(out, "dinitial", (S, W - 1, D), dt, dev)
        pws, ws_bytes, workspace = _workspace(workspace, need, dev)
        layer_call("kda_short_conv_backward", desc, px, pw, pb, p0, cu, pdy, pdf, pdx, pdw, pdb, pdi, pws, ws_bytes,
                   st)
    return out


# ---------------------------------------------------------------- selective scan
def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, lead):
    """Checks shared by the scan's calls: the descriptor's lengths and distances, and the input addresses."""
    torch = _torch()
    dev, ty, f32 = _device(x, "x"), x.dtype, torch.float32
    rows, ch = x.shape[:lead], x.shape[-1]
    if A.dim() != 2 or B.dim() != lead + 2:
        raise ValueError(f"A must be [D, N] and B, C {lead + 2}-dimensional ([.., G, N])")
    N, G = A.shape[1], B.shape[-2]
    px, ld_x = _rows("x", x, dev, ty, x.shape, lead)
    pdt, ld_dt = _rows("dt", dt, dev, ty, x.shape, lead)
    pA = _like("A", A, dev, f32, (ch, N))
    pB, ld_b = _rows("B", B, dev, ty, (*rows, G, N), lead)
    pC, ld_c = _rows("C", C, dev, ty, (*rows, G, N), lead)
    pD = _like("D", D, dev, f32, (ch,))
    pz, ld_z = (None, 0) if z is None else _rows("z", z, dev, ty, x.shape, lead)
    pb = _like("dt_bias", dt_bias, dev, f32, (ch,))
    return dev, ty, N, G, (ld_x, ld_dt, ld_z, ld_b, ld_c), (px, pdt, pA, pB, pC, pD, pz, pb)


def selective_scan_workspace_bytes(B: int, T: int, D: int, N: int, dtype, G: int = 1, n_seqs: int = 0) -> int:
    """Device workspace one selective_scan_forward call of this shape needs."""
    return layer_workspace_size("kda_selective_scan", ScanDesc(*_ints(B, T, D, N, G, n_seqs), _code(dtype), 1))


def selective_scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, h0=None, cu_seqlens=None,
                           dt_softplus: bool = True, o=None, ht=None, workspace=None,
                           output_final_state: bool = True, validate_cu: bool = True, stream=None):
    """Selective state space scan over whole sequences (kda_selective_scan_forward):
    delta = softplus(dt + dt_bias), h_t = exp(delta_t A) h_{t-1} + delta_t B_t x_t,
    o_t = (sum_n C_t h_t + D x_t) z_t sigmoid(z_t).

    x, dt, z: [B, T, D] (bf16 or fp32; z may be None: no gate), or packed
    [1, sum of lengths, D] with cu_seqlens (int32 [n + 1]); A: fp32 [D, N], N
    up to 64; B, C: [B, T, G, N], group g serving channels g D / G ..;
    D, dt_bias: fp32 [D] or None; h0: fp32 [S, D, N] or None (zeros).
    dt_softplus False takes dt + dt_bias as delta itself.  Returns (o, ht
    fp32 [S, D, N], or None when output_final_state is False).  ht must not be
    h0's memory."""
    torch = _torch()
    dev, ty, N, G, lds, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, 2)
    Bt, T, ch = x.shape
    n_seqs, S, cu = _sequences(cu_seqlens, Bt, T, dev, validate_cu)
    p0 = _like("h0", h0, dev, torch.float32, (S, ch, N))
    desc = ScanDesc(*_ints(Bt, T, ch, N, G, n_seqs), _code(ty), dt_softplus, *lds)
    with _On(dev, stream) as st:
        need = layer_workspace_size("kda_selective_scan", desc)
        o, po = _new(o, x, "o", dev, (Bt, T, ch))
        ph = None
        if ht is not None or output_final_state:
            ht, ph = _new(ht, x, "ht", dev, (S, ch, N), torch.float32)
        pws, ws_bytes, workspace = _workspace(workspace, need, dev) if need else (None, 0, None)
        layer_call("kda_selective_scan_forward", desc, *ptrs, p0, cu, po, ph, pws, ws_bytes, st)
    return o, ht


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, *, dt_softplus: bool = True, o=None,
                        stream=None):
    """One token for each of S sequences: x, dt, z [S, D], B, C [S, G, N];
    state fp32 [S, D, N] is updated in place (kda_selective_scan_step).
    Returns o [S, D]."""
    torch = _torch()
    dev, ty, N, G, lds, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, 1)
    S, ch = x.shape
    ps = _like("state", state, dev, torch.float32, (S, ch, N))
    if S == 0:
        return x.new_empty((0, ch)) if o is None else o
    desc = ScanDesc(*_ints(S, 1, ch, N, G, 0), _code(ty), dt_softplus, *lds)
    with _On(dev, stream) as st:
        o, po = _new(o, x, "o", dev, (S, ch))
        layer_call("kda_selective_scan_step", desc, *ptrs, ps, po, st)
    _written(state)
    return o


def selective_scan_backward(x, dt, A, B, C, do, D=None, z=None, dt_bias=None, *, h0=None, dht=None, cu_seqlens=None,
                            dt_softplus: bool = True, out=None, workspace=None, validate_cu: bool = True,
                            stream=None) -> dict:
    """Gradients of <do, o> + <dht, ht> for selective_scan_forward with the
    same inputs (kda_selective_scan_backward): a dict with dx, ddt, dz, dB, dC
    in x's dtype and dA, dD, ddt_bias, dh0 in fp32, each in its input's shape;
    dz, dD, ddt_bias and dh0 are None where that input is.  `out` may supply
    those tensors."""
    torch = _torch()
    f32 = torch.float32
    dev, ty, N, G, lds, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, 2)
    Bt, T, ch = x.shape
    n_seqs, S, cu = _sequences(cu_seqlens, Bt, T, dev, validate_cu)
    p0 = _like("h0", h0, dev, f32, (S, ch, N))
    pdo = _like("do", do, dev, ty, (Bt, T, ch))
    pdht = _like("dht", dht, dev, f32, (S, ch, N))
    desc = ScanDesc(*_ints(Bt, T, ch, N, G, n_seqs), _code(ty), dt_softplus, *lds)
    need = layer_workspace_size("kda_selective_scan_backward", desc)
    out = dict(out or {})
    with _On(dev, stream) as st:
        pdx = _out(out, "dx", (Bt, T, ch), ty, dev)
        pddt = _out(out, "ddt", (Bt, T, ch), ty, dev)
        pdA = _out(out, "dA", (ch, N), f32, dev)
        pdB = _out(out, "dB", (Bt, T, G, N), ty, dev)
        pdC = _out(out, "dC", (Bt, T, G, N), ty, dev)
        pdD = pdz = pdb = pdh = None
        if D is not None or out.setdefault("dD", None) is not None:
            pdD = _out(out, "dD", (ch,), f32, dev)
        if z is None:
            out["dz"] = None
        else:
            pdz = _out(out, "dz", (Bt, T, ch), ty, dev)
        if dt_bias is not None or out.setdefault("ddt_bias", None) is not None:
            pdb = _out(out, "ddt_bias", (ch,), f32, dev)
        if h0 is not None or out.setdefault("dh0", None) is not None:
            pdh = _out(out, "dh0", (S, ch, N), f32, dev)
        pws, ws_bytes, workspace = _workspace(workspace, need, dev)
        layer_call("kda_selective_scan_backward", desc, *ptrs, p0, cu, pdo, pdht, pdx, pddt, pdA, pdB, pdC, pdD, pdz,
                   pdb, pdh, pws, ws_bytes, st)
    return out


# ---------------------------------------------------------------- norm of queries and keys
def _norm_inputs(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, interleaved, q_scale):
    torch = _torch()
    dev, ty, f32 = _device(q, "q"), q.dtype, torch.float32
    if q.dim() < 3 or k.dim() != q.dim():
        raise ValueError("q and k must be [.., heads, d] with the same token dims")
    if norm not in _NORMS:
        raise ValueError(f"norm must be 'l2' or 'rms', got {norm!r}")
    if (positions is None) != (inv_freq is None):
        raise ValueError("a rotation needs both positions and inv_freq")
    lead = q.dim() - 2
    rows, Hq, d, Hk = q.shape[:lead], q.shape[-2], q.shape[-1], k.shape[-2]
    pq, ld_q = _rows("q", q, dev, ty, q.shape, lead)
    pk, ld_k = _rows("k", k, dev, ty, (*rows, Hk, d), lead)
    rot, pp, pf = 0, None, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        pf = _like("inv_freq", inv_freq, dev, f32, (rot // 2,))
        pp = _like("positions", positions, dev, torch.int32, rows)
        if rot == 0:
            pp = pf = None
    tokens = 1
    for s in rows:
        tokens *= s
    desc = NormDesc(*_ints(tokens, Hq, Hk, d, rot), _code(ty), _NORMS[norm], interleaved, eps, q_scale, ld_q, ld_k)
    return dev, ty, desc, (pq, pk, _like("q_weight", q_weight, dev, f32, (d,)),
                           _like("k_weight", k_weight, dev, f32, (d,)), pp, pf)


def qk_norm_forward(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, norm="l2",
                    eps: float = 1e-6, interleaved: bool = False, q_scale: float = 1.0, q_out=None, k_out=None,
                    stream=None):
    """Norm of every query and key head, and the rotation by the token's
    position, in one pass (kda_qk_norm_forward).

    q: [.., Hq, d], k: [.., Hk, d] (bf16 or fp32) with the same token dims, d
    even.  norm "l2" makes unit vectors (what chunk_forward and decode_step
    take), "rms" divides by the root mean square; then the weights (fp32 [d] or
    None).  positions: int32 of the token dims, inv_freq: fp32 [R / 2]: the
    first R channels are turned in pairs by positions * inv_freq; the pairs
    are channels (i, i + R / 2), or (2 i, 2 i + 1) when interleaved.  q_scale
    multiplies q's output.  Returns (q_out, k_out), contiguous."""
    dev, ty, desc, ptrs = _norm_inputs(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, interleaved, q_scale)
    with _On(dev, stream) as st:
        q_out, pq = _new(q_out, q, "q_out", dev, q.shape)
        k_out, pk = _new(k_out, k, "k_out", dev, k.shape)
        layer_call("kda_qk_norm_forward", desc, *ptrs, pq, pk, st)
    return q_out, k_out


def qk_norm_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, norm="l2",
                     eps: float = 1e-6, interleaved: bool = False, q_scale: float = 1.0, out=None, workspace=None,
                     stream=None) -> dict:
    """Gradients of <dq_out, q_out> + <dk_out, k_out> for qk_norm_forward with
    the same inputs (kda_qk_norm_backward): a dict with dq, dk in q's dtype and
    dq_weight, dk_weight fp32 [d] (None without the weight, unless `out`
    supplies the tensor)."""
    torch = _torch()
    dev, ty, desc, ptrs = _norm_inputs(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, interleaved, q_scale)
    pdq, pdk = _like("dq_out", dq_out, dev, ty, q.shape), _like("dk_out", dk_out, dev, ty, k.shape)
    need = layer_workspace_size("kda_qk_norm_backward", desc)
    out = dict(out or {})
    d = q.shape[-1]
    with _On(dev, stream) as st:
        pq, pk = _out(out, "dq", q.shape, ty, dev), _out(out, "dk", k.shape, ty, dev)
        pwq = pwk = None
        if q_weight is not None or out.setdefault("dq_weight", None) is not None:
            pwq = _out(out, "dq_weight", (d,), torch.float32, dev)
        if k_weight is not None or out.setdefault("dk_weight", None) is not None:
            pwk = _out(out, "dk_weight", (d,), torch.float32, dev)
        pws, ws_bytes, workspace = _workspace(workspace, need, dev)
        layer_call("kda_qk_norm_backward", desc, *ptrs, pdq, pdk, pq, pk, pwq, pwk, pws, ws_bytes, st)
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

    class ShortConv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation, validate_cu):
            y, final = short_conv_forward(x, weight, bias, initial_state=initial_state, cu_seqlens=cu_seqlens,
                                          activation=activation, validate_cu=validate_cu,
                                          **cleared(cu_seqlens, validate_cu, y=x))
            ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
            ctx.activation, ctx.validated = activation, validate_cu
            ctx.set_materialize_grads(False)
            return y, final

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy, dfinal):
            x, weight, bias, init, cu = ctx.saved_tensors
            g = short_conv_backward(x, weight, full(dy, x), bias, initial_state=init,
                                    dfinal=None if dfinal is None else dfinal.contiguous(), cu_seqlens=cu,
                                    activation=ctx.activation, validate_cu=False, out=cleared(cu, ctx.validated, dx=x))
            return g["dx"], g["dweight"], g["dbias"], g["dinitial"], None, None, None

    class SelectiveScan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dt_softplus, validate_cu):
            o, ht = selective_scan_forward(x, dt, A, B, C, D, z, dt_bias, h0=h0, cu_seqlens=cu_seqlens,
                                           dt_softplus=dt_softplus, validate_cu=validate_cu,
                                           **cleared(cu_seqlens, validate_cu, o=x))
            ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens)
            ctx.dt_softplus, ctx.validated = dt_softplus, validate_cu
            ctx.set_materialize_grads(False)
            return o, ht

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, do, dht):
            x, dt, A, B, C, D, z, dt_bias, h0, cu = ctx.saved_tensors
            g = selective_scan_backward(x, dt, A, B, C, full(do, x), D, z, dt_bias, h0=h0,
                                        dht=None if dht is None else dht.contiguous(), cu_seqlens=cu,
                                        dt_softplus=ctx.dt_softplus, validate_cu=False,
                                        out=cleared(cu, ctx.validated, dx=x, ddt=dt, dB=B, dC=C, dz=z))
            return (g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddt_bias"], g["dh0"], None,
                    None, None)

    class QKNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, options):
            ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
            ctx.options = options
            ctx.set_materialize_grads(False)
            return qk_norm_forward(q, k, q_weight, k_weight, positions, inv_freq, **options)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dq_out, dk_out):
            q, k, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
            g = qk_norm_backward(q, k, full(dq_out, q), full(dk_out, k), q_weight, k_weight, positions, inv_freq,
                                 **ctx.options)
            return g["dq"], g["dk"], g["dq_weight"], g["dk_weight"], None, None, None

    _FUNCTIONS = ShortConv, SelectiveScan, QKNorm
    return _FUNCTIONS


def short_conv(x, weight, bias=None, *, initial_state=None, cu_seqlens=None, activation="silu",
               validate_cu: bool = True):
    """short_conv_forward as a differentiable PyTorch operation: returns
    (y, final_state); its backward is short_conv_backward."""
    return _functions()[0].apply(x, weight, bias, initial_state, cu_seqlens, activation, validate_cu)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, h0=None, cu_seqlens=None,
                   dt_softplus: bool = True, validate_cu: bool = True):
    """selective_scan_forward as a differentiable PyTorch operation: returns
    (o, ht); its backward is selective_scan_backward."""
    return _functions()[1].apply(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dt_softplus, validate_cu)


def qk_norm(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, norm="l2", eps: float = 1e-6,
            interleaved: bool = False, q_scale: float = 1.0):
    """qk_norm_forward as a differentiable PyTorch operation: returns (q_out,
    k_out); its backward is qk_norm_backward (q, k and the weights)."""
    options = dict(norm=norm, eps=eps, interleaved=interleaved, q_scale=q_scale)
    return _functions()[2].apply(q, k, q_weight, k_weight, positions, inv_freq, options)
