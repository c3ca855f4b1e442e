"""Bounded waits of the dense attention kernels, made to run out on purpose by a
copy that is told to expect 16 bytes more than it brings: the call comes back
with QUEST_DEVERR_WAIT_TIMEOUT and the next one is right."""

import numpy as np
import pytest

from tests._cases import F16, F32, dev_i32, gpu_cache, gpu_table, np_of
from tests._dense_ref import attention, check_attention
from tests.test_gpu_dense import _rows_case

pytestmark = pytest.mark.gpu

WAIT_TIMEOUT, LIMIT = 0x8, 2000


def _recovers(call, check):
    import query_aware_sparse_gb300 as qs
    qs.device_error()
    qs.test_step_fault(2, LIMIT)
    try:
        call()
        err = qs.device_error()
    finally:
        qs.test_step_fault(0, 0)
    assert err & WAIT_TIMEOUT, err
    out = call()
    assert qs.device_error() == 0
    check(*out)


@pytest.mark.parametrize("dtype,group,d", [(F16, 2, 128), (F16, 8, 64), (F32, 2, 64)])
def test_decode_wait_runs_out(dtype, group, d):
    import query_aware_sparse_gb300 as qs
    case = _rows_case(201, [2000, 300, 40], [1, 1, 1], h_kv=2, group=group, d=d, S=16, dtype=dtype)
    t = case["table"]
    cache, table, q = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(t), case["q"].cuda()
    ref = attention(np_of(case["q"]), np_of(case["k_pool"]), np_of(case["v_pool"]), t.page_indptr, t.page_indices,
                    t.seq_lens, np.arange(4), group)
    _recovers(lambda: qs.dense_decode_attn(cache, table, q, group),
              lambda o, l: check_attention(np_of(o), np_of(l), ref, 0.0, 0.0, 2000))


@pytest.mark.parametrize("lens,rows,d", [([300, 40], [300, 2], 128), ([200], [200], 64),
                                         ([9000], [9], 128), ([9000], [200], 128)])
def test_prefill_wait_runs_out(lens, rows, d):
    """Blocks of one and of two row tiles, whole and cut along the keys."""
    import query_aware_sparse_gb300 as qs
    case = _rows_case(202, lens, rows, h_kv=1, group=2, d=d, S=16)
    t = case["table"]
    cache, table, q = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(t), case["q"].cuda()
    ref = attention(np_of(case["q"]), np_of(case["k_pool"]), np_of(case["v_pool"]), t.page_indptr, t.page_indices,
                    t.seq_lens, case["q_indptr"], 2)
    ind = dev_i32(case["q_indptr"])
    _recovers(lambda: qs.prefill_attn(cache, table, q, 2, ind),
              lambda o, l: check_attention(np_of(o), np_of(l), ref, 2.0 ** -11, 2.0 ** -11, max(lens)))
