"""Rows of prompt attention beyond what the host passes."""

import numpy as np
import pytest
import torch

from tests._cases import F16, F32, dev_i32, gpu_cache, gpu_table, np_of
from tests._dense_ref import attention, check_attention
from tests.test_gpu_dense import HALF16, _rows_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("n", [1, 100, 150, 201])
def test_more_rows_in_the_table_than_passed(n, dtype):
    """q_indptr names more rows than n_q: the first n_q are computed, at their places,
    and no per-row input behind them is read."""
    import query_aware_sparse_gb300 as qs
    lens, rows = [200, 90], [150, 60]
    case = _rows_case(600, lens, rows, h_kv=2, group=2, d=64, S=16, dtype=dtype)
    docs = np.concatenate([np.arange(L - r, L) // 50 * 50 for L, r in zip(lens, rows)]).astype(np.int32)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    out, lse = qs.prefill_attn(cache, table, case["q"][:n].cuda(), 2, dev_i32(case["q_indptr"]),
                               mods=qs.ScoreMods(doc_starts=dev_i32(docs[:n])))
    assert qs.device_error() == 0
    t = case["table"]
    ref = attention(np_of(case["q"]), np_of(case["k_pool"]), np_of(case["v_pool"]), t.page_indptr, t.page_indices,
                    t.seq_lens, case["q_indptr"], 2, doc_starts=docs)
    half = HALF16 if dtype == F16 else 0.0
    check_attention(np_of(out), np_of(lse), {k: v[:n] for k, v in ref.items()}, half, half, 200)
