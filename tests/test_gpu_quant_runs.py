"""Decode over the E4M3 cache in equal runs, in the shapes whose heads stand in
the tensor core's columns twice, against the fp64 forms on the stored numbers."""

import pytest

from tests._quant_ref import quant_case
from tests.test_gpu_quant_decode import _dense, _sparse

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,S,group", [(128, 32, 4), (128, 32, 1), (128, 32, 2), (128, 16, 2), (128, 16, 4), (64, 16, 4), (64, 32, 2)])
def test_equal_runs_of_packed_heads(d, S, group):
    """Tables and lists too long for a cluster per unit."""
    case = quant_case(430 + S + group, [24000, 31, 0, 9000], h_kv=1, group=group, d=d, S=S)
    _dense(case)
    _dense(case, ["cap", "alibi", "doc"], seed=3)
    _dense(case, ["window"], seed=4)
    _sparse(case, 700, seed=1, drop=0.1)
