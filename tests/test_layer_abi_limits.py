"""Refusals of the operators around the recurrence at the edges of their
sizes, on the CPU: what a kernel would read although there are no tokens.
Each call carries an argument that has to be refused, so none reaches a launch
(the pointers are fake addresses)."""
import pytest

from gated_delta_rule_105_amd._lib import KDA_ERR_INVALID_ARGUMENT as INV
from gated_delta_rule_105_amd._lib import ConvDesc, ScanDesc
from test_layer_abi import call, desc


@pytest.mark.parametrize("name,kind,param", [("kda_selective_scan_forward", ScanDesc, "A"),
                                             ("kda_selective_scan_backward", ScanDesc, "A"),
                                             ("kda_short_conv_backward", ConvDesc, "weight")])
@pytest.mark.parametrize("packed", [False, True])
def test_null_parameters_without_tokens(name, kind, param, packed):
    """Batches without tokens still write states and gradients, by kernels that read the parameters."""
    d = desc(kind, T=0, **(dict(B=1, n_seqs=2) if packed else {}))
    assert call(name, d=d, **{param: None}) == INV
