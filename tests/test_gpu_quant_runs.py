"""Decode over the E4M3 cache in equal runs, in the shapes whose heads stand in
the tensor core's columns twice, against the fp64 forms on the stored numbers."""

import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("d,S,group", [(64, 16, 2), (128, 32, 1), (128, 16, 8)])
def test_more_units_than_the_device_holds(d, S, group):
    """Lists on both sides of the border between a CTA per unit, several waves of
    them, and equal runs; some empty, some shorter than k."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(d + S)
    batch = 3 * sms // 8 + 9                          # of 8 heads: more than three CTAs per SM
    border = 4 * (12 + batch * 8 * group // 150)      # pages
    lens = rng.integers(0, (border + 8) * S, batch)
    lens[3], lens[5] = 0, (border + 8) * S
    case = quant_case(440 + group, lens.tolist(), h_kv=8, group=group, d=d, S=S)
    for k in (9, border, border + 1):
        _sparse(case, k, seed=k, drop=0.1)


@pytest.mark.parametrize("d,S,group", [(128, 16, 4), (64, 16, 8)])
def test_clusters_look_up_their_tiles_more_than_once(d, S, group):
    """Lists and a table of more tiles than the 32 that a warp of a cluster takes
    from them at a time: 16 requests of 8 heads leave three CTAs per unit."""
    rng = np.random.default_rng(group)
    lens = rng.integers(0, 40, 16)
    lens[2], lens[9] = 600 * S - 5, 0
    case = quant_case(450 + group, lens.tolist(), h_kv=8, group=group, d=d, S=S)
    assert 32 * 12 < case["table"].nnz <= 64 * 12
    _dense(case)
    _dense(case, ["cap", "window", "doc"], seed=6)
    _sparse(case, 590, seed=2, drop=0.4)              # holes among the slots of a look


@pytest.mark.parametrize("d,S,group", [(128, 16, 2), (64, 32, 8)])
def test_a_batch_padded_with_empty_requests(d, S, group):
    """A table of few pages for more units than the device holds at once: a CTA
    each, most of them without a token."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(group)
    lens = np.zeros(4 * sms, int)
    lens[rng.permutation(len(lens))[:30]] = rng.integers(1, S + 1, 30)
    lens[-1] = 9 * S + 1
    case = quant_case(460 + group, lens.tolist(), h_kv=1, group=group, d=d, S=S)
    assert case["table"].nnz <= 4 * 12
    _dense(case)
    _dense(case, ["alibi", "prefix"], seed=7)
