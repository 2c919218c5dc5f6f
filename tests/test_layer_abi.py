"""C-ABI checks of the operators around the recurrence that need no GPU:
workspace sizes, and every refusal.  Each call below carries at least one
invalid argument, so none reaches a launch (the pointers are fake addresses)."""
import ctypes

import pytest

from gated_delta_rule_105_amd import _lib
from gated_delta_rule_105_amd._lib import (KDA_ACT_SILU, KDA_DTYPE_BF16, KDA_ERR_INVALID_ARGUMENT,
                                           KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE_TOO_SMALL, KDA_NORM_RMS,
                                           KDA_NORM_UNIT, KDA_OK, ConvDesc, NormDesc, ScanDesc)

GB = 1 << 30
INV, UNS, SMALL = KDA_ERR_INVALID_ARGUMENT, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE_TOO_SMALL

# pointer arguments of each call, in order; those that may be NULL; those written
CALLS = {
    "kda_short_conv_forward": (ConvDesc, "x weight bias init cu y fin", "bias init fin", "y fin"),
    "kda_short_conv_step": (ConvDesc, "x weight bias state y", "bias", "state y"),
    "kda_short_conv_backward": (ConvDesc, "x weight bias init cu dy dfin dx dw db dinit", "bias init dfin db dinit",
                                "dx dw db dinit"),
    "kda_selective_scan_forward": (ScanDesc, "x dt A B C skip z bias h0 cu o ht", "skip z bias h0 ht", "o ht"),
    "kda_selective_scan_step": (ScanDesc, "x dt A B C skip z bias state o", "skip z bias", "state o"),
    "kda_selective_scan_backward": (ScanDesc, "x dt A B C skip z bias h0 cu do dht dx ddt dA dB dC dskip dz dbias dh0",
                                    "skip z bias h0 dht dskip dbias dh0", "dx ddt dA dB dC dskip dz dbias dh0"),
    "kda_qk_norm_forward": (NormDesc, "q k wq wk pos freq qo ko", "wq wk", "qo ko"),
    "kda_qk_norm_backward": (NormDesc, "q k wq wk pos freq dqo dko dq dk dwq dwk", "wq wk dwq dwk", "dq dk dwq dwk"),
}


def desc(kind, **kw):
    base = {ConvDesc: dict(B=2, T=100, D=256, width=4, n_seqs=0, dtype=KDA_DTYPE_BF16, activation=KDA_ACT_SILU, ld_x=0),
            ScanDesc: dict(B=2, T=100, D=256, N=16, G=2, n_seqs=0, dtype=KDA_DTYPE_BF16, softplus=1, ld_x=0, ld_dt=0,
                           ld_z=0, ld_b=0, ld_c=0),
            NormDesc: dict(n_tokens=200, Hq=8, Hk=2, d=128, rot=64, dtype=KDA_DTYPE_BF16, norm=KDA_NORM_RMS,
                           interleaved=0, eps=1e-6, q_scale=1.0, ld_q=0, ld_k=0)}[kind]
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
    tail = [ws, ws_bytes, None] if _lib.LAYER_CALLS[name][2] else [None]
    return getattr(_lib.load(), name)(ctypes.byref(d) if d is not False else None, *args.values(), *tail)


def test_mirrors_have_the_header_layout():
    assert ctypes.sizeof(ConvDesc) == 40 and ConvDesc.ld_x.offset == 32
    assert ctypes.sizeof(ScanDesc) == 72 and ScanDesc.ld_x.offset == 32
    assert ctypes.sizeof(NormDesc) == 56 and NormDesc.ld_q.offset == 40 and NormDesc.eps.offset == 32
    for name, (kind, n, _) in _lib.LAYER_CALLS.items():
        assert kind is CALLS[name][0] and n == len(CALLS[name][1].split())


@pytest.mark.parametrize("name", CALLS)
def test_null_arguments(name):
    _, names, optional, _ = CALLS[name]
    for n in names.split():
        if n not in optional.split() and n != "cu":
            assert call(name, **{n: None}) == INV, n
    assert call(name, d=False) == INV


@pytest.mark.parametrize("name", CALLS)
def test_misaligned_arguments(name):
    kind, names, _, _ = CALLS[name]
    d = desc(kind, **({"T": 1} if name.endswith("_step") else {}))
    for i, n in enumerate(names.split()):
        if n != "cu":
            assert call(name, d=d, **{n: address(i) + 1}) == INV, n
    if "n_seqs" in dict(kind._fields_) and not name.endswith("_step"):
        d = desc(kind, B=1, n_seqs=3)
        assert call(name, d=d, cu=address(40) + 2) == INV


@pytest.mark.parametrize("name", CALLS)
def test_overlapping_outputs(name):
    """An output may be neither an input's memory nor another output's."""
    _, names, _, written = CALLS[name]
    all_names = [n for n in names.split() if n != "cu"]
    where = {n: address(i) for i, n in enumerate(names.split())}
    for out in written.split():
        for other in all_names:
            if other != out:
                assert call(name, **{out: where[other]}) == INV, (out, other)
        if _lib.LAYER_CALLS[name][2] and (name != "kda_selective_scan_forward"):
            assert call(name, ws=where[out] // 256 * 256) == INV, out


@pytest.mark.parametrize("name,kw", [
    ("kda_short_conv_backward", {}), ("kda_selective_scan_backward", {}), ("kda_qk_norm_backward", {}),
    ("kda_selective_scan_forward", dict(B=1, T=4096))])
def test_workspace(name, kw):
    kind = CALLS[name][0]
    d = desc(kind, **kw)
    size = ctypes.c_size_t(0)
    sizer = getattr(_lib.load(), name.replace("_scan_forward", "_scan") + "_workspace_size")
    assert sizer(ctypes.byref(d), ctypes.byref(size)) == KDA_OK and size.value > 0
    assert sizer(ctypes.byref(d), None) == INV
    assert sizer(None, ctypes.byref(size)) == INV
    assert call(name, d=d, ws_bytes=size.value - 1) == SMALL
    assert call(name, d=d, ws=None) == INV
    assert call(name, d=d, ws=500 * 64 * GB + 64) == INV


def test_workspace_sizes():
    def size(name, d):
        out = ctypes.c_size_t(0)
        st = getattr(_lib.load(), name + "_workspace_size")(ctypes.byref(d), ctypes.byref(out))
        return st, out.value
    # rows that fill the device need no state between slots; no tokens need none either
    assert size("kda_selective_scan", desc(ScanDesc, B=64, D=1024, G=1)) == (KDA_OK, 0)
    assert size("kda_selective_scan", desc(ScanDesc, T=0)) == (KDA_OK, 0)
    assert size("kda_short_conv_backward", desc(ConvDesc, T=0)) == (KDA_OK, 0)
    # a state of every slot, and its sum of delta
    st, n = size("kda_selective_scan", desc(ScanDesc, B=1, T=65536, D=64, G=1))
    assert st == KDA_OK and n % (64 * 17 * 4) % 256 == 0 and n >= 100 * 64 * 17 * 4
    assert size("kda_qk_norm_backward", desc(NormDesc)) == (KDA_OK, 2 * 256 * 128 * 4)


BAD_CONV = [(dict(B=0), INV), (dict(T=-1), INV), (dict(D=0), INV), (dict(width=0), INV), (dict(width=1), UNS),
            (dict(width=5), UNS), (dict(n_seqs=-1), INV), (dict(n_seqs=3), INV), (dict(dtype=2), INV),
            (dict(dtype=-1), INV), (dict(activation=2), INV), (dict(ld_x=255), INV), (dict(ld_x=-1), INV),
            (dict(B=65536, T=65536), UNS), (dict(ld_x=2 ** 62), INV), (dict(D=2 ** 24), UNS)]
BAD_SCAN = [(dict(B=0), INV), (dict(T=-1), INV), (dict(D=0), INV), (dict(N=0), INV), (dict(N=65), UNS),
            (dict(G=0), INV), (dict(G=3), INV), (dict(n_seqs=-1), INV), (dict(n_seqs=2), INV), (dict(dtype=7), INV),
            (dict(ld_x=255), INV), (dict(ld_dt=1), INV), (dict(ld_z=-5), INV), (dict(ld_b=31), INV),
            (dict(ld_c=31), INV), (dict(B=65536, T=65536), UNS), (dict(ld_c=2 ** 62), INV),
            (dict(B=1, T=2 ** 30, D=2 ** 20, G=1), UNS)]
BAD_NORM = [(dict(n_tokens=-1), INV), (dict(Hq=0), INV), (dict(Hk=0), INV), (dict(d=0), INV), (dict(rot=-2), INV),
            (dict(rot=130), INV), (dict(rot=63), INV), (dict(d=127, rot=64), UNS), (dict(d=514), UNS),
            (dict(dtype=3), INV), (dict(norm=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
            (dict(eps=float("inf")), INV), (dict(q_scale=float("nan")), INV), (dict(q_scale=float("inf")), INV),
            (dict(ld_q=1023), INV), (dict(ld_k=100), INV), (dict(Hq=70000), UNS), (dict(rot=0), INV)]


@pytest.mark.parametrize("name", CALLS)
def test_bad_descriptors(name):
    kind = CALLS[name][0]
    step = {"T": 1} if name.endswith("_step") else {}
    for kw, code in {ConvDesc: BAD_CONV, ScanDesc: BAD_SCAN, NormDesc: BAD_NORM}[kind]:
        assert call(name, d=desc(kind, **dict(step, **kw))) in ((code, INV) if step else (code,)), kw


@pytest.mark.parametrize("name", ["kda_short_conv_step", "kda_selective_scan_step"])
def test_steps_take_one_token(name):
    kind = CALLS[name][0]
    assert call(name, d=desc(kind, T=2)) == INV
    assert call(name, d=desc(kind, T=0)) == INV
    assert call(name, d=desc(kind, T=1, B=1, n_seqs=1)) == INV


@pytest.mark.parametrize("name", ["kda_short_conv_forward", "kda_short_conv_backward", "kda_selective_scan_forward",
                                  "kda_selective_scan_backward"])
def test_offsets_go_with_packed_sequences(name):
    kind = CALLS[name][0]
    assert call(name, d=desc(kind, B=1, n_seqs=3), cu=None) == INV
    assert call(name, d=desc(kind), cu=address(40)) == INV


def test_rotation_arguments_go_together():
    for name in ("kda_qk_norm_forward", "kda_qk_norm_backward"):
        assert call(name, pos=None) == INV
        assert call(name, freq=None) == INV
        assert call(name, d=desc(NormDesc, rot=0, norm=KDA_NORM_UNIT), pos=None) == INV


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import gated_delta_rule_105_amd as kda
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="device tensor"):
        kda.short_conv_forward(x, w)
    with pytest.raises(ValueError, match="device tensor"):
        kda.short_conv_step(x[0], w, torch.zeros(4, 3, 8))
    with pytest.raises(ValueError, match="device tensor"):
        kda.selective_scan_forward(x, x, torch.zeros(8, 2), torch.zeros(1, 4, 1, 2), torch.zeros(1, 4, 1, 2))
    with pytest.raises(ValueError, match="device tensor"):
        kda.qk_norm_forward(x.view(1, 4, 1, 8), x.view(1, 4, 1, 8))


def test_binding_refuses_lengths_past_32_bits():
    """The descriptors' lengths are 32-bit; a longer one would wrap to a short call."""
    torch = pytest.importorskip("torch")
    import gated_delta_rule_105_amd as kda
    with pytest.raises(ValueError, match="2\\^31"):
        kda.selective_scan_workspace_bytes(1, 2 ** 32 + 64, 64, 16, torch.bfloat16)
    meta = torch.empty(1, 2 ** 32 + 5, 1, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        kda.layer._conv_desc(meta, None, 1, meta.shape[1], 1, 4, 0, "silu", 0)
