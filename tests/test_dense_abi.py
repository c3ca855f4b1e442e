"""Argument checks of the dense-layer calls (rotating append, dense decode and
prompt attention): they return before any CUDA call, so no GPU is needed."""

import ctypes

import pytest
import torch

FAKE = 0x10000                      # never dereferenced: validation fails first
F = ctypes.c_float(0.0)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def q():
    from query_aware_sparse_gb300 import build
    build.build()
    import query_aware_sparse_gb300 as q
    return q


def _cache(q, **over):
    v = dict(k=FAKE, v=FAKE, s=FAKE, n=8, h=2, S=16, d=128, dt=q.QUEST_F16, f8=0)
    v.update(over)
    return q.QuestCache(*v.values())


def _pages(q, batch=1, nnz=8, seq=FAKE):
    return q.QuestPages(FAKE, FAKE, seq, batch, nnz)


def _append(qs_, cache=None, pages=None, rope=None, **over):
    q = qs_
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, n=1, group=4, ind=FAKE, before=FAKE,
             out=FAKE + 4096)
    a.update(over)
    by = ctypes.byref
    rope = q.QuestRope(FAKE, None, 128, 0) if rope is None else rope
    return q.lib().quest_rope_append_kv(by(cache or _cache(q)), by(pages or _pages(q)), by(rope),
                                        *a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(group=3), UNSUPPORTED),
    (dict(n=-1), INVALID),
    (dict(qs=1016), INVALID),            # shorter than the row
    (dict(qs=1028), INVALID),            # rows off their 16-byte boundary
    (dict(ks=248), INVALID),
    (dict(ks=260), INVALID),
    (dict(vs=8), INVALID),
    (dict(q=None), INVALID),             # q_out without q
    (dict(out=None), INVALID),
    (dict(q=FAKE + 2), INVALID),
    (dict(k=FAKE + 8), INVALID),
    (dict(v=None), INVALID),
    (dict(ind=None), INVALID),
    (dict(before=None), INVALID),
    (dict(out=FAKE, qs=2048), INVALID),  # in place only without gaps
])
def test_append_refuses(q, over, status):
    assert _append(q, **over) == status


@pytest.mark.parametrize("rope,status", [
    ((FAKE, None, 0, 0), UNSUPPORTED), ((FAKE, None, 24, 0), UNSUPPORTED),
    ((FAKE, None, 144, 0), UNSUPPORTED), ((FAKE, None, 64, 2), INVALID),
    ((None, None, 64, 0), INVALID), ((FAKE + 4, None, 64, 0), INVALID)])
def test_append_refuses_rotation(q, rope, status):
    assert _append(q, rope=q.QuestRope(*rope)) == status


@pytest.mark.parametrize("over,status", [
    (dict(d=96), UNSUPPORTED), (dict(S=24), UNSUPPORTED), (dict(dt=7), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=FAKE + 2), INVALID), (dict(h=0), INVALID),
    (dict(dt=0, f8=1), UNSUPPORTED)])
def test_every_call_checks_the_cache(q, over, status):
    by, L, c = ctypes.byref, q.lib(), _cache(q, **over)
    assert _append(q, cache=c) == status
    assert L.quest_dense_decode_attn(by(c), by(_pages(q)), FAKE, 4, None, FAKE, FAKE, F, FAKE,
                                     1 << 30, None) == status
    assert L.quest_prefill_attn(by(c), by(_pages(q)), FAKE, 4, FAKE, 3, None, FAKE, FAKE, F, FAKE,
                                1 << 30, None) == status


@pytest.mark.parametrize("mods,status", [
    ((None, None, None, -1.0, 0), INVALID), ((None, None, None, float("nan"), 0), INVALID),
    ((None, None, None, float("inf"), 0), INVALID), ((None, None, None, 1e-7, 0), INVALID),
    ((None, None, None, 0.0, -4), INVALID)])
def test_attention_refuses_mods(q, mods, status):
    by, L, c, m = ctypes.byref, q.lib(), _cache(q), q.QuestScoreMods(*mods)
    assert L.quest_dense_decode_attn(by(c), by(_pages(q)), FAKE, 4, by(m), FAKE, FAKE, F, FAKE,
                                     1 << 30, None) == status
    assert L.quest_prefill_attn(by(c), by(_pages(q)), FAKE, 4, FAKE, 3, by(m), FAKE, FAKE, F, FAKE,
                                1 << 30, None) == status


def test_attention_refuses_arguments(q):
    by, L, c, p = ctypes.byref, q.lib(), _cache(q), _pages(q)

    def dec(qq=FAKE, group=4, out=FAKE, ws=FAKE, size=1 << 30, pages=p):
        return L.quest_dense_decode_attn(by(c), by(pages), qq, group, None, out, None, F, ws, size, None)

    def pre(qq=FAKE, group=4, ind=FAKE, n=3, out=FAKE, ws=FAKE, size=1 << 30, pages=p):
        return L.quest_prefill_attn(by(c), by(pages), qq, group, ind, n, None, out, None, F, ws, size, None)

    for f in (dec, pre):
        assert f(qq=None) == INVALID and f(qq=FAKE + 2) == INVALID
        assert f(out=None) == INVALID and f(out=FAKE + 4) == INVALID
        assert f(group=3) == UNSUPPORTED and f(group=16) == UNSUPPORTED
        assert f(ws=None) == WORKSPACE and f(ws=FAKE + 8) == WORKSPACE and f(size=0) == WORKSPACE
        assert f(pages=_pages(q, seq=None)) == INVALID
    assert pre(ind=None) == INVALID and pre(n=-1) == INVALID
    assert dec(pages=_pages(q, batch=(1 << 19) + 1)) == UNSUPPORTED


def test_empty_calls_are_no_ops(q):
    by, L, c = ctypes.byref, q.lib(), _cache(q)
    none = q.QuestPages(None, None, None, 0, 0)
    assert _append(q, n=0) == 0 and _append(q, pages=none) == 0
    assert L.quest_dense_decode_attn(by(c), by(none), None, 4, None, None, None, F, None, 0, None) == 0
    assert L.quest_prefill_attn(by(c), by(none), None, 4, None, 3, None, None, None, F, None, 0, None) == 0
    assert L.quest_prefill_attn(by(c), by(_pages(q)), None, 4, None, 0, None, None, None, F, None, 0, None) == 0


def test_workspace_sizes(q):
    L = q.lib()
    for dt in (q.QUEST_F16, q.QUEST_F32):
        assert L.quest_dense_decode_workspace_size(1, 2048, 32, 1, 128, 16, dt) > 0
        assert L.quest_prefill_workspace_size(1, 16, 2048, 32, 1, 128, 16, dt) > 0
    for bad in ((0, 8, 2, 4, 128, 16, 1), (1, -1, 2, 4, 128, 16, 1), (1, 8, 0, 4, 128, 16, 1),
                (1, 8, 2, 3, 128, 16, 1), (1, 8, 2, 4, 96, 16, 1), (1, 8, 2, 4, 128, 24, 1),
                (1, 8, 2, 4, 128, 16, 5)):
        assert L.quest_dense_decode_workspace_size(*bad) == 0
        assert L.quest_prefill_workspace_size(bad[0], 4, *bad[1:]) == 0


def test_binding_refuses_tensors(q):
    """The Python calls check types, shapes, devices and layout first."""
    pool = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    cache = q.PagedCache(pool, pool.clone(), torch.zeros((4, 2, 2, 64), dtype=torch.float16))
    table = q.PageTable(torch.tensor([0, 4], dtype=torch.int32), torch.arange(4, dtype=torch.int32),
                        torch.tensor([50], dtype=torch.int32))
    i32 = torch.tensor([0, 1], dtype=torch.int32)
    x = torch.zeros((1, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.dense_decode_attn(cache, table, x, 1)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.prefill_attn(cache, table, x, 1, i32)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.rope_append_kv(cache, table, x, x, x, i32, i32[:1], torch.ones(32, dtype=torch.float64), 1)
    dev = x.get_device()
    q._expect("x", x, torch.float16, (1, 2, 64), dev)
    for bad in (x.float(), x[0], x.expand(3, 2, 64)):
        with pytest.raises(ValueError, match="x must be"):
            q._expect("x", bad, torch.float16, (1, 2, 64), dev)
    with pytest.raises(ValueError, match="x must be"):
        q._expect("x", x, torch.float16, (1, 2, 64), 5)
    wide = torch.zeros((3, 4, 64), dtype=torch.float16)
    part = wide[:, :2]
    assert q._expect_rows("part", part, torch.float16, (3, 2, 64), dev) == 256
    assert q._expect_rows("part", part[:1], torch.float16, (1, 2, 64), dev) == 128
    assert q._expect_rows("part", wide[:, 3:], torch.float16, (3, 1, 64), dev) == 256
    with pytest.raises(ValueError, match="contiguous"):
        q._expect("part", part, torch.float16, (3, 2, 64), dev)
    for bad in (wide[:, ::2], wide[:1, :2].expand(3, 2, 64), wide[..., ::2].repeat(1, 1, 2).transpose(1, 2)[:, :2],
                part.float()):
        with pytest.raises(ValueError, match="part must be"):
            q._expect_rows("part", bad, torch.float16, (3, 2, 64), dev)
    m = q.ScoreMods(doc_starts=i32)
    with pytest.raises(ValueError, match="doc_starts"):
        m.check(2, 1, 1, dev)


def test_binding_refuses_places(q, monkeypatch):
    """Streams, workspaces and page tables of another device; windows beyond 32 bits."""
    class Stream:
        device_index, cuda_stream = 1, 77
    assert q._raw_stream(Stream, 1) == 77
    with pytest.raises(ValueError, match="stream must be"):
        q._raw_stream(Stream, 0)
    ws = torch.zeros(64, dtype=torch.uint8)
    q._expect_workspace(ws, ws.get_device())
    for bad, dev in ((ws, 0), (ws[::2], ws.get_device())):
        with pytest.raises(ValueError, match="workspace must be"):
            q._expect_workspace(bad, dev)
    class On:
        def __init__(self, dev):
            self.dev = dev

        def get_device(self):
            return self.dev
    assert q._common_device(On(1), On(1), On(1)) == 1
    assert q._common_device(On(0), On(1), On(0)) == q._common_device(On(0), On(0), On(-1)) == -1
    pool = torch.zeros((1, 1, 16, 64), dtype=torch.float16)
    cache, i32 = q.PagedCache(pool, pool, pool[:, :, :2]), torch.tensor([0, 1], dtype=torch.int32)
    table = q.PageTable(i32, i32[:1], i32[1:])
    assert cache.device_index == table.device_index == -1
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    cache.device_index = 0
    with pytest.raises(ValueError, match="page table must be"):
        q._current(cache, table)
    table.device_index = 0
    assert q._current(cache, table) == 0
    for bad in (1 << 31, (1 << 32) + 5, -(1 << 31)):
        with pytest.raises(ValueError, match="window"):
            q.ScoreMods(window=bad)
    assert q.ScoreMods(window=(1 << 31) - 1).c.window == (1 << 31) - 1


def test_attention_refuses_pools_beyond_a_coordinate(q):
    by, L, p = ctypes.byref, q.lib(), _pages(q)
    rows = (1 << 31) // 16
    for n, h, refused in ((rows // 2, 2, True), (rows // 2 - 1, 2, False), (1 << 30, 1 << 20, True)):
        c = _cache(q, n=n, h=h)
        got = (L.quest_dense_decode_attn(by(c), by(p), FAKE, 4, None, FAKE, FAKE, F, None, 0, None),
               L.quest_prefill_attn(by(c), by(p), None, 4, FAKE, 3, None, FAKE, FAKE, F, FAKE, 1 << 30, None))
        want = (UNSUPPORTED, UNSUPPORTED) if refused else (WORKSPACE, INVALID)
        assert got == want, (n, h)


def test_frequencies(q):
    f = q.rope_frequencies(64, base=500000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    assert float(f[0]) == 1.0 and abs(float(f[16]) - 500000.0 ** -0.5) < 1e-15
