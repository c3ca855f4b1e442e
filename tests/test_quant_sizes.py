"""quest_quant_decode_workspace_size gives 0 for exactly the sizes that the
calls refuse as unsupported (no GPU is needed: nothing is launched)."""

import ctypes

import pytest

FAKE = 0x10000                      # never dereferenced: validation fails first
UNSUPPORTED, WORKSPACE = -2, -3
by = ctypes.byref


@pytest.mark.parametrize("batch,h_kv,group,fits", [
    (1, 1, 1, True), (524288, 4095, 1, True), (524288, 511, 8, True), (1023, 1 << 18, 8, True),
    (524289, 1, 1, False), (524288, 4096, 1, False), (524288, 512, 8, False), (1024, 1 << 18, 8, False),
    (1, 1 << 30, 2, False),
])
@pytest.mark.parametrize("S,d", [(16, 64), (32, 128)])
def test_size_and_call_agree(batch, h_kv, group, fits, S, d):
    from query_aware_sparse_gb300 import build
    build.build()
    import query_aware_sparse_gb300 as q
    assert fits == (batch <= 524288 and batch * h_kv * group < 1 << 31)
    assert (q.quant_decode_workspace_size(batch, h_kv, group, d, S) > 0) == fits
    cache = q.QuestQuantCache(FAKE, FAKE, 8, h_kv, S, d, 0)
    pages = q.QuestPages(FAKE, FAKE, FAKE, batch, 8)
    scale = ctypes.c_float(0.0)
    # without a workspace what is supported gets no further
    want = WORKSPACE if fits else UNSUPPORTED
    assert q.lib().quest_quant_dense_decode_attn(by(cache), by(pages), FAKE, group, None, FAKE, FAKE, scale, None, 0, None) == want
    assert q.lib().quest_quant_sparse_decode_attn(by(cache), by(pages), FAKE, group, FAKE, FAKE, 4, FAKE, FAKE, scale, None, 0,
                                                  None) == want
