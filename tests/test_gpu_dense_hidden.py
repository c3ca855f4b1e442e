"""What no row may see has no part in a result: the same bits whatever stands in
slots without a token, in shared memory before the call, and in the rows of
other requests."""

import numpy as np
import pytest
import torch

from tests._cases import F16, F32, dev_i32, gpu_cache, gpu_table
from tests.test_gpu_dense import _rows_case

pytestmark = pytest.mark.gpu

LENS, ROWS = [70, 33, 200, 5], [70, 3, 129, 1]
MODS = [dict(softcap=50.0), dict(softcap=3.0), dict(softcap=50.0, alibi=True), dict(softcap=50.0, window=20), dict()]


def _mods(kw, hq):
    import query_aware_sparse_gb300 as qs
    kw = dict(kw)
    slopes = 2.0 ** -torch.arange(1, hq + 1, device="cuda").float() if kw.pop("alibi", False) else None
    return qs.ScoreMods(alibi_slopes=slopes, **kw)


def _slots(case, value):
    """The pools with `value` in every slot without a token."""
    t, S = case["table"], case["S"]
    kept = torch.zeros((t.n_phys, S), dtype=torch.bool)
    for r, L in enumerate(t.seq_lens):
        for p in range(-(-int(L) // S)):
            kept[int(t.page_indices[t.page_indptr[r] + p]), :max(0, min(S, int(L) - p * S))] = True
    keep = kept[:, None, :, None].expand_as(case["k_pool"])
    return [torch.where(keep, case[x], torch.full_like(case[x], value)) for x in ("k_pool", "v_pool")]


def _spoil(d, dtype, value):
    """Prompts of large keys: what they leave in shared memory is found by the next call."""
    import query_aware_sparse_gb300 as qs
    pool = torch.full((16, 4, 16, d), value, dtype=dtype, device="cuda")
    cache = qs.PagedCache(pool, pool, torch.zeros((16, 4, 2, d), dtype=dtype, device="cuda"))
    table = qs.PageTable(dev_i32(np.arange(0, 17 * 16, 16)), dev_i32(np.tile(np.arange(16), 16)), dev_i32([256] * 16))
    q = torch.full((16 * 256, 4, d), value, dtype=dtype, device="cuda")
    qs.prefill_attn(cache, table, q, 1, dev_i32(np.arange(0, 17 * 256, 256)))


def _prefill(case, cache, table, q, mods):
    import query_aware_sparse_gb300 as qs
    return qs.prefill_attn(cache, table, q, 2, dev_i32(case["q_indptr"]), mods=mods)


def _decode(case, cache, table, q, mods):
    import query_aware_sparse_gb300 as qs
    last = torch.as_tensor(case["q_indptr"][1:] - 1, device="cuda").long()
    return qs.dense_decode_attn(cache, table, q[last].contiguous(), 2, mods=mods)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", MODS)
@pytest.mark.parametrize("call", [_prefill, _decode])
def test_slots_without_a_token(call, kw, d, dtype):
    import query_aware_sparse_gb300 as qs
    case = _rows_case(401, LENS, ROWS, h_kv=2, group=2, d=d, S=16, dtype=dtype)
    table, q = gpu_table(case["table"]), case["q"].cuda()
    mods, first = _mods(kw, 4), None
    for value in (0.0, float("nan"), 6e4, -6e4, float("inf")):
        cache = gpu_cache(*_slots(case, value), case["summary"])
        _spoil(d, dtype, 200.0 if value == 0.0 else 0.01)
        got = call(case, cache, table, q, mods)
        first = first or got
        for a, b in zip(first, got):
            assert torch.equal(a, b), value
    assert qs.device_error() == 0


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", MODS)
def test_rows_of_other_requests(kw, d, dtype):
    """A request's rows next to large queries, of other requests and behind the last."""
    import query_aware_sparse_gb300 as qs
    case = _rows_case(402, LENS, ROWS, h_kv=2, group=2, d=d, S=16, dtype=dtype)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    ind, mods = dev_i32(case["q_indptr"]), _mods(kw, 4)
    q = torch.cat([case["q"], torch.zeros((9, 4, d), dtype=dtype)]).cuda()
    n = sum(ROWS)
    out, lse = qs.prefill_attn(cache, table, q, 2, ind, mods=mods)
    for r in range(len(LENS)):
        a, b = int(case["q_indptr"][r]), int(case["q_indptr"][r + 1])
        other = torch.full_like(q, 100.0)
        other[a:b] = q[a:b]
        got = qs.prefill_attn(cache, table, other, 2, ind, mods=mods)
        assert torch.equal(got[0][a:b], out[a:b]) and torch.equal(got[1][a:b], lse[a:b]), r
    assert torch.isfinite(lse[:n]).all() and qs.device_error() == 0
