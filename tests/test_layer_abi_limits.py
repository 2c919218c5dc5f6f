"""Refusals of the operators around the recurrence at the edges of their
sizes, on the CPU: what a kernel would read although there are no tokens, and
batches whose launches no grid holds.  Each call carries an argument that has to be refused, so none reaches a launch
(the pointers are fake addresses)."""
import ctypes

import pytest

from gated_delta_rule_105_amd import _lib
from gated_delta_rule_105_amd._lib import KDA_DTYPE_BF16, ConvDesc, NormDesc, ScanDesc
from gated_delta_rule_105_amd._lib import KDA_ERR_INVALID_ARGUMENT as INV
from gated_delta_rule_105_amd._lib import KDA_ERR_UNSUPPORTED as UNS
from test_layer_abi import call, desc


@pytest.mark.parametrize("name,kind,param", [("kda_selective_scan_forward", ScanDesc, "A"),
                                             ("kda_selective_scan_backward", ScanDesc, "A"),
                                             ("kda_short_conv_backward", ConvDesc, "weight")])
@pytest.mark.parametrize("packed", [False, True])
def test_null_parameters_without_tokens(name, kind, param, packed):
    """Batches without tokens still write states and gradients, by kernels that read the parameters."""
    d = desc(kind, T=0, **(dict(B=1, n_seqs=2) if packed else {}))
    assert call(name, d=d, **{param: None}) == INV


@pytest.mark.parametrize("name,kind,kw", [
    ("kda_short_conv_forward", ConvDesc, dict(B=1, T=1200000000, D=1, dtype=KDA_DTYPE_BF16)),
    ("kda_selective_scan_forward", ScanDesc, dict(B=32768, T=1, D=4096, G=1024)),
    ("kda_selective_scan_backward", ScanDesc, dict(B=1, T=2 ** 20, D=1024, G=256)),
    ("kda_qk_norm_forward", NormDesc, dict(n_tokens=100000000, Hq=1, Hk=1))])
def test_launches_past_the_grid_are_refused(name, kind, kw):
    """A launch has less than 2^32 threads along its first dimension: refused before anything runs, and by the
    workspace's size likewise."""
    d = desc(kind, **kw)
    assert call(name, d=d, ws_bytes=1 << 62) == UNS
    size = {"kda_selective_scan_forward": "kda_selective_scan",
            "kda_selective_scan_backward": "kda_selective_scan_backward"}.get(name)
    if size:
        out = ctypes.c_size_t(0)
        assert getattr(_lib.load(), size + "_workspace_size")(ctypes.byref(d), ctypes.byref(out)) == UNS
