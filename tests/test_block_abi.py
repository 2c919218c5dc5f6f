"""C-ABI checks of linear attention and the norms at a block's end that need
no GPU: workspace sizes, and every refusal.  Each call below carries at least
one invalid argument, so none reaches a launch (the pointers are fake
addresses)."""
import ctypes

import pytest

from gated_delta_rule_105_amd import _lib
from gated_delta_rule_105_amd._lib import (KDA_ACT_NONE, KDA_ACT_SIGMOID, KDA_DECAY_HEAD, KDA_DECAY_NONE,
                                           KDA_DECAY_TOKEN, KDA_DTYPE_BF16, KDA_DTYPE_F32, KDA_ERR_INVALID_ARGUMENT,
                                           KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE_TOO_SMALL, KDA_OK, GatedNormDesc,
                                           LinearDesc, ResidualNormDesc)

GB = 1 << 30
INV, UNS, SMALL = KDA_ERR_INVALID_ARGUMENT, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE_TOO_SMALL

# pointer arguments of each call, in order; those that may be NULL; those written
CALLS = {
    "kda_linear_attn_forward": (LinearDesc, "q k v g h0 cu o ht", "h0 ht", "o ht"),
    "kda_linear_attn_step": (LinearDesc, "q k v g state o", "", "state o"),
    "kda_linear_attn_backward": (LinearDesc, "q k v g h0 cu do dht dq dk dv dg dh0", "h0 dht dg dh0",
                                 "dq dk dv dg dh0"),
    "kda_gated_norm_forward": (GatedNormDesc, "x gate w y", "w", "y"),
    "kda_gated_norm_backward": (GatedNormDesc, "x gate w dy dx dgate dw", "w dw", "dx dgate dw"),
    "kda_residual_norm_forward": (ResidualNormDesc, "x res w c y total", "w c", "y total"),
    "kda_residual_norm_backward": (ResidualNormDesc, "x total w c dy dtotal dx dres dw dc", "w c dtotal dx dw dc",
                                   "dx dres dw dc"),
}


def desc(kind, **kw):
    base = {LinearDesc: dict(B=2, T=1000, Hq=2, H=4, d_k=64, d_v=128, n_seqs=0, dtype=KDA_DTYPE_BF16,
                             decay=KDA_DECAY_TOKEN, scale=0.5, ld_q=0, ld_k=0, ld_v=0, ld_g=0),
            GatedNormDesc: dict(n_tokens=200, H=8, d=128, dtype=KDA_DTYPE_BF16, activation=KDA_ACT_SIGMOID, eps=1e-6,
                                ld_x=0, ld_gate=0),
            ResidualNormDesc: dict(n_tokens=200, D=1024, dtype=KDA_DTYPE_F32, scale=1.0, eps=1e-6, ld_x=0,
                                   ld_residual=0)}[kind]
    return kind(**dict(base, **kw))


def address(i):
    return (i + 1) * 64 * GB


def call(name, d=None, ws=500 * 64 * GB, ws_bytes=1 << 40, **ptrs):
    """A call with distinct fake addresses but for `ptrs`."""
    kind, names, _, _ = CALLS[name]
    d = desc(kind, T=1) if d is None and name.endswith("_step") else desc(kind) if d is None else d
    args = {n: address(i) for i, n in enumerate(names.split())}
    if "cu" in args and (d is False or d.n_seqs == 0):
        args["cu"] = None
    assert set(ptrs) <= set(args)
    args.update(ptrs)
    tail = [ws, ws_bytes, None] if _lib.BLOCK_CALLS[name][2] else [None]
    return getattr(_lib.load(), name)(ctypes.byref(d) if d is not False else None, *args.values(), *tail)


def size_of(name, d):
    out = ctypes.c_size_t(0)
    name = name.replace("kda_linear_attn_forward", "kda_linear_attn")
    return getattr(_lib.load(), name + "_workspace_size")(ctypes.byref(d), ctypes.byref(out)), out.value


def test_mirrors_have_the_header_layout():
    assert ctypes.sizeof(LinearDesc) == 72 and LinearDesc.scale.offset == 36 and LinearDesc.ld_q.offset == 40
    assert ctypes.sizeof(GatedNormDesc) == 40 and GatedNormDesc.eps.offset == 20 and GatedNormDesc.ld_x.offset == 24
    assert ctypes.sizeof(ResidualNormDesc) == 40 and ResidualNormDesc.ld_x.offset == 24
    for name, (kind, n, _) in _lib.BLOCK_CALLS.items():
        assert kind is CALLS[name][0] and n == len(CALLS[name][1].split())


@pytest.mark.parametrize("name", CALLS)
def test_null_arguments(name):
    _, names, optional, _ = CALLS[name]
    for n in names.split():
        if n not in optional.split() and n != "cu" and (n, name) != ("x", "kda_residual_norm_backward"):
            assert call(name, **{n: None}) == INV, n
    assert call(name, d=False) == INV


def test_channel_gradients_need_x():
    assert call("kda_residual_norm_backward", x=None) == INV


@pytest.mark.parametrize("name", CALLS)
def test_misaligned_arguments(name):
    kind, names, _, _ = CALLS[name]
    d = desc(kind, **({"T": 1} if name.endswith("_step") else {}))
    for i, n in enumerate(names.split()):
        if n != "cu":
            assert call(name, d=d, **{n: address(i) + 1}) == INV, n
    if kind is LinearDesc:
        d = desc(kind, decay=KDA_DECAY_HEAD, **({"T": 1} if name.endswith("_step") else {}))
        more = dict(dg=None) if name.endswith("backward") else {}
        assert call(name, d=d, g=address(3) + 2, **more) == INV  # fp32
        if not name.endswith("_step"):
            assert call(name, d=desc(kind, B=1, n_seqs=3), cu=address(40) + 2) == INV


@pytest.mark.parametrize("name", CALLS)
def test_overlapping_outputs(name):
    """An output may be neither an input's memory, nor another output's, nor the workspace."""
    _, names, _, written = CALLS[name]
    all_names = [n for n in names.split() if n != "cu"]
    where = {n: address(i) for i, n in enumerate(names.split())}
    for out in written.split():
        for other in all_names:
            if other != out:
                assert call(name, **{out: where[other]}) == INV, (out, other)
        if _lib.BLOCK_CALLS[name][2]:
            assert call(name, ws=where[out]) == INV, out


@pytest.mark.parametrize("name", [n for n in CALLS if _lib.BLOCK_CALLS[n][2]])
def test_workspace(name):
    kind = CALLS[name][0]
    st, need = size_of(name, desc(kind))
    assert st == KDA_OK and need > 0
    sizer = getattr(_lib.load(), name.replace("attn_forward", "attn") + "_workspace_size")
    assert sizer(ctypes.byref(desc(kind)), None) == INV
    assert sizer(None, ctypes.byref(ctypes.c_size_t(0))) == INV
    assert call(name, ws_bytes=need - 1) == SMALL
    assert call(name, ws=None) == INV
    assert call(name, ws=500 * 64 * GB + 64) == INV


def test_workspace_sizes():
    # rows that fill the device need no state between slots; no tokens need none either
    assert size_of("kda_linear_attn_forward", desc(LinearDesc, B=64, Hq=8, H=8)) == (KDA_OK, 0)
    assert size_of("kda_linear_attn_forward", desc(LinearDesc, T=0)) == (KDA_OK, 0)
    assert size_of("kda_gated_norm_backward", desc(GatedNormDesc, n_tokens=0)) == (KDA_OK, 0)
    # gradients of shared queries and keys by head, in fp32
    st, alone = size_of("kda_linear_attn_backward", desc(LinearDesc, Hq=4))
    st2, shared = size_of("kda_linear_attn_backward", desc(LinearDesc))
    assert st == st2 == KDA_OK and shared - alone == 2 * 2000 * 4 * 64 * 4


BAD_LINEAR = [(dict(B=0), INV), (dict(T=-1), INV), (dict(Hq=0), INV), (dict(H=0), INV), (dict(Hq=3), INV),
              (dict(d_k=0), INV), (dict(d_v=-1), INV), (dict(d_k=129), UNS), (dict(d_v=200), UNS),
              (dict(n_seqs=-1), INV), (dict(n_seqs=3), INV), (dict(dtype=2), INV), (dict(decay=3), INV),
              (dict(decay=-1), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
              (dict(ld_q=127), INV), (dict(ld_k=-1), INV), (dict(ld_v=511), INV), (dict(ld_g=3), INV),
              (dict(ld_v=2 ** 62), INV), (dict(B=65536, T=65536), UNS), (dict(B=2 ** 21, T=1, H=2048), UNS),
              (dict(ld_q=2 ** 22 + 1), UNS), (dict(ld_k=2 ** 22 + 1), UNS), (dict(ld_v=2 ** 22 + 1), UNS),
              (dict(ld_g=2 ** 22 + 1), UNS), (dict(T=1, Hq=1, H=2 ** 16, d_v=128), UNS)]
BAD_GATED = [(dict(n_tokens=-1), INV), (dict(H=0), INV), (dict(d=0), INV), (dict(d=8193), UNS), (dict(H=70000), UNS),
             (dict(dtype=2), INV), (dict(activation=KDA_ACT_NONE), INV), (dict(activation=3), INV),
             (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(ld_x=1023), INV),
             (dict(ld_gate=-5), INV), (dict(ld_gate=2 ** 62), INV), (dict(n_tokens=2 ** 30), UNS)]
BAD_RESIDUAL = [(dict(n_tokens=-1), INV), (dict(D=0), INV), (dict(D=8193), UNS), (dict(dtype=-1), INV),
                (dict(scale=float("nan")), INV), (dict(scale=float("-inf")), INV), (dict(eps=-1.0), INV),
                (dict(eps=float("nan")), INV), (dict(ld_x=1023), INV), (dict(ld_residual=1), INV),
                (dict(ld_x=2 ** 62), INV)]


@pytest.mark.parametrize("name", CALLS)
def test_bad_descriptors(name):
    kind = CALLS[name][0]
    step = {"T": 1} if name.endswith("_step") else {}
    for kw, code in {LinearDesc: BAD_LINEAR, GatedNormDesc: BAD_GATED, ResidualNormDesc: BAD_RESIDUAL}[kind]:
        assert call(name, d=desc(kind, **dict(step, **kw)), ws_bytes=1 << 62) in ((code, INV) if step else (code,)), kw


def test_steps_take_one_token():
    for kw in (dict(T=2), dict(T=0), dict(T=1, B=1, n_seqs=1)):
        assert call("kda_linear_attn_step", d=desc(LinearDesc, **kw)) == INV


@pytest.mark.parametrize("name", ["kda_linear_attn_forward", "kda_linear_attn_backward"])
def test_offsets_go_with_packed_sequences(name):
    assert call(name, d=desc(LinearDesc, B=1, n_seqs=3), cu=None) == INV
    assert call(name, cu=address(40)) == INV


@pytest.mark.parametrize("name", ["kda_linear_attn_forward", "kda_linear_attn_step", "kda_linear_attn_backward"])
def test_decays_go_with_their_kind(name):
    step = {"T": 1} if name.endswith("_step") else {}
    more = dict(dg=None) if name.endswith("backward") else {}
    assert call(name, d=desc(LinearDesc, decay=KDA_DECAY_NONE, **step), **more) == INV
    assert call(name, d=desc(LinearDesc, decay=KDA_DECAY_HEAD, **step), g=None, **more) == INV
    if more:  # a fixed decay has no gradient
        assert call(name, d=desc(LinearDesc, decay=KDA_DECAY_HEAD)) == INV
        assert call(name, d=desc(LinearDesc, decay=KDA_DECAY_NONE), g=None) == INV
        # a fixed decay is read for the states of empty sequences too
        assert call(name, d=desc(LinearDesc, T=0, decay=KDA_DECAY_HEAD), g=None, **more) == INV


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    import gated_delta_rule_105_amd as kda
    x = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        kda.linear_attn_forward(x, x, x)
    with pytest.raises(ValueError, match="device tensor"):
        kda.linear_attn_step(x[0], x[0], x[0], torch.zeros(4, 2, 8, 8))
    with pytest.raises(ValueError, match="device tensor"):
        kda.gated_norm_forward(x, x)
    with pytest.raises(ValueError, match="device tensor"):
        kda.residual_norm_forward(x, x)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.linear_attn_workspace_bytes(1, 2 ** 32 + 64, 2, 64, 64, torch.bfloat16)
