"""Every call that reads or writes fp16 or fp32 pages answers a QuantCache with
the same TypeError, before anything is enqueued (CPU tensors: no GPU is needed)."""

import pytest
import torch


@pytest.fixture(scope="module")
def case():
    from query_aware_sparse_gb300 import build
    build.build()
    import query_aware_sparse_gb300 as qs
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    cache = qs.QuantCache.empty(4, 2, 16, 64, device="cpu")
    table = qs.PageTable(i32(0, 4), i32(0, 1, 2, 3), i32(50))
    return qs, cache, table, torch.zeros(1, 2, 64, dtype=torch.float16), torch.zeros(1, 2, 2, dtype=torch.int32), i32


CALLS = {
    "append_kv": lambda qs, c, t, q, sel, i32: qs.append_kv(c, t, q, q, i32(0, 1), i32(49), stream=1),
    "sparse_decode_attn": lambda qs, c, t, q, sel, i32: qs.sparse_decode_attn(
        c, t, q, 1, sel, sel, 2, workspace=torch.zeros(16, dtype=torch.uint8), stream=1),
    "sparse_decode_attn_noalloc": lambda qs, c, t, q, sel, i32: qs.sparse_decode_attn_noalloc(c, t, q, 1, sel, sel, 2, stream=1),
    "union_decode_attn": lambda qs, c, t, q, sel, i32: qs.union_decode_attn(
        c, t, q, 1, sel, 2, workspace=torch.zeros(16, dtype=torch.uint8), stream=1),
    "recall_diagnostics": lambda qs, c, t, q, sel, i32: qs.recall_diagnostics(c, t, q, 1, sel, 2, 4, stream=1),
    "DecodeStep": lambda qs, c, t, q, sel, i32: qs.DecodeStep(c, t, 1, 2),
    "DecodeStep_on_a_device": lambda qs, c, t, q, sel, i32: qs.DecodeStep(c, t, 1, 2, device="cpu"),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_quant_cache_is_refused(case, name):
    qs, *args = case
    with pytest.raises(TypeError, match="quant_read_kv"):
        CALLS[name](qs, *args)
