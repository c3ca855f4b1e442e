"""Argument checks of the normed append and of the E4M3 cache's calls: they
return before any CUDA call, so no GPU is needed."""

import ctypes

import pytest
import torch

FAKE = 0x10000                      # never dereferenced: validation fails first
F = ctypes.c_float(0.0)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
by = ctypes.byref


@pytest.fixture(scope="module")
def q():
    from query_aware_sparse_gb300 import build
    build.build()
    import query_aware_sparse_gb300 as q
    return q


def _plain(q, **over):
    v = dict(k=FAKE, v=FAKE, s=FAKE, n=8, h=2, S=16, d=128, dt=q.QUEST_F16, f8=0)
    v.update(over)
    return q.QuestCache(*v.values())


def _quant(q, **over):
    v = dict(pool=FAKE, s=FAKE, n=8, h=2, S=16, d=128, f8=0)
    v.update(over)
    return q.QuestQuantCache(*v.values())


def _pages(q, batch=1, nnz=8, seq=FAKE):
    return q.QuestPages(FAKE, FAKE, seq, batch, nnz)


def _norm(q, **over):
    v = dict(qw=FAKE, kw=FAKE, qp=0, kp=0, eps=1e-6)
    v.update(over)
    return q.QuestQKNorm(*v.values())


def _append(qs_, quant, cache=None, pages=None, rope="full", norm="all", **over):
    q = qs_
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, n=1, group=4, ind=FAKE, before=FAKE, out=FAKE + 4096)
    a.update(over)
    rope = q.QuestRope(FAKE, None, 128, 0) if rope == "full" else rope
    norm = _norm(q) if norm == "all" else norm
    ref = lambda x: None if x is None else by(x)  # noqa: E731
    cache = cache or (_quant(q) if quant else _plain(q))
    call = q.lib().quest_quant_append_kv if quant else q.lib().quest_norm_rope_append_kv
    return call(by(cache), by(pages or _pages(q)), ref(rope), ref(norm), *a.values(), None)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("over,status", [
    (dict(group=3), UNSUPPORTED),
    (dict(n=-1), INVALID),
    (dict(qs=1016), INVALID),            # shorter than the row
    (dict(qs=1028), INVALID),            # rows off their 16-byte boundary
    (dict(ks=248), INVALID),
    (dict(vs=260), INVALID),
    (dict(q=None), INVALID),             # q_out without q
    (dict(out=None), INVALID),
    (dict(q=FAKE + 2), INVALID),
    (dict(k=FAKE + 8), INVALID),
    (dict(v=None), INVALID),
    (dict(ind=None), INVALID),
    (dict(before=None), INVALID),
    (dict(out=FAKE, qs=2048), INVALID),  # in place only without gaps
])
def test_append_refuses(q, quant, over, status):
    assert _append(q, quant, **over) == status


@pytest.mark.parametrize("quant", [False, True])
def test_append_refuses_norms_and_rotations(q, quant):
    for over, status in ((dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
                         (dict(eps=float("inf")), INVALID), (dict(eps=1e-45), INVALID), (dict(qp=2), INVALID),
                         (dict(kp=-1), INVALID), (dict(qw=FAKE + 4), INVALID), (dict(kw=FAKE + 8), INVALID)):
        assert _append(q, quant, norm=_norm(q, **over)) == status, over
    for rope, status in ((q.QuestRope(FAKE, None, 8, 0), UNSUPPORTED), (q.QuestRope(FAKE, None, 136, 0), UNSUPPORTED),
                         (q.QuestRope(FAKE, None, 24, 0), UNSUPPORTED), (q.QuestRope(FAKE, None, 64, 2), INVALID),
                         (q.QuestRope(None, None, 64, 0), INVALID), (q.QuestRope(FAKE + 4, None, 64, 0), INVALID)):
        assert _append(q, quant, rope=rope) == status
    # nothing to do to a query
    assert _append(q, quant, rope=None, norm=_norm(q, qw=None)) == INVALID
    assert _append(q, quant, norm=None, n=0) == (0 if quant else INVALID)
    assert _append(q, True, rope=None, norm=None) == INVALID
    assert _append(q, True, rope=None, norm=None, q=None, out=None, n=0) == 0
    assert _append(q, quant, n=0) == 0
    assert _append(q, quant, pages=_pages(q, batch=0)) == 0
    assert _append(q, quant, pages=_pages(q, batch=-1)) == INVALID


def test_caches_are_checked(q):
    lib = q.lib()
    ws = 1 << 30

    def calls(c):
        return [_append(q, True, cache=c), lib.quest_quant_read_kv(by(c), by(_pages(q)), FAKE, FAKE, 8, None, None),
                lib.quest_quant_sparse_decode_attn(by(c), by(_pages(q)), FAKE, 4, FAKE, FAKE, 4, FAKE, FAKE, F, FAKE, ws, None),
                lib.quest_quant_dense_decode_attn(by(c), by(_pages(q)), FAKE, 4, None, FAKE, FAKE, F, FAKE, ws, None)]
    for over, status in ((dict(pool=None), INVALID), (dict(s=None), INVALID), (dict(pool=FAKE + 8), INVALID),
                         (dict(s=FAKE + 2), INVALID), (dict(n=0), INVALID), (dict(h=0), INVALID), (dict(f8=2), INVALID),
                         (dict(d=96), UNSUPPORTED), (dict(S=8), UNSUPPORTED), (dict(S=64), UNSUPPORTED)):
        assert calls(_quant(q, **over)) == [status] * 4, over


def test_read_refuses(q):
    read = lambda pages=None, k=FAKE, v=FAKE, n=8: q.lib().quest_quant_read_kv(  # noqa: E731
        by(_quant(q)), by(pages or _pages(q)), k, v, n, None, None)
    assert read(k=None) == read(v=None) == read(k=FAKE + 2) == read(v=FAKE + 8) == read(n=-1) == INVALID
    assert read(pages=_pages(q, seq=None)) == read(pages=_pages(q, nnz=-1)) == INVALID
    assert read(pages=_pages(q, batch=0)) == 0
    big = _quant(q, h=1 << 20)
    assert q.lib().quest_quant_read_kv(by(big), by(_pages(q, nnz=1 << 20)), FAKE, FAKE, 8, None, None) == UNSUPPORTED


def test_decode_refuses(q):
    need = q.quant_decode_workspace_size(1, 2, 4, 128, 16)
    lib = q.lib()

    def sparse(pages=None, qq=FAKE, group=4, sl=FAKE, sp=FAKE, k=4, out=FAKE, ws=FAKE, size=need):
        return lib.quest_quant_sparse_decode_attn(by(_quant(q)), by(pages or _pages(q)), qq, group, sl, sp, k, out, FAKE, F, ws,
                                                  size, None)

    def dense(pages=None, qq=FAKE, group=4, mods=None, out=FAKE, ws=FAKE, size=need):
        return lib.quest_quant_dense_decode_attn(by(_quant(q)), by(pages or _pages(q)), qq, group,
                                                 None if mods is None else by(mods), out, FAKE, F, ws, size, None)
    for call in (sparse, dense):
        assert call(qq=None) == call(out=None) == call(qq=FAKE + 8) == call(out=FAKE + 4) == INVALID
        assert call(ws=None) == call(ws=FAKE + 8) == call(size=need - 1) == WORKSPACE
        assert call(pages=_pages(q, batch=0)) == 0
        assert call(pages=_pages(q, batch=524289)) == UNSUPPORTED
        assert call(pages=_pages(q, seq=None)) == INVALID
    assert sparse(group=3) == sparse(k=0) == sparse(sl=None) == sparse(sp=None) == INVALID
    assert dense(group=3) == UNSUPPORTED
    for m in (q.QuestScoreMods(None, None, None, 1e-7, 0), q.QuestScoreMods(None, None, None, -1.0, 0),
              q.QuestScoreMods(None, None, None, float("inf"), 0), q.QuestScoreMods(None, None, None, 0.0, -1)):
        assert dense(mods=m) == INVALID
    wide = _quant(q, h=1 << 20)
    many = _pages(q, batch=1024)
    assert lib.quest_quant_dense_decode_attn(by(wide), by(many), FAKE, 8, None, FAKE, FAKE, F, FAKE, 1 << 40, None) == UNSUPPORTED


def test_sizes(q):
    assert q.quant_page_bytes(16, 128) == 4128 and q.quant_page_bytes(32, 64) == 4160
    assert q.quant_page_bytes(8, 128) == q.quant_page_bytes(16, 96) == 0
    assert q.quant_decode_workspace_size(0, 2, 4, 128, 16) == q.quant_decode_workspace_size(1, 2, 3, 128, 16) == 0
    assert q.quant_decode_workspace_size(1, 2, 4, 96, 16) == q.quant_decode_workspace_size(524289, 1, 1, 64, 16) == 0
    small, large = (q.quant_decode_workspace_size(b, 2, 4, 128, 16) for b in (1, 64))
    assert 0 < small < large


def test_python_wrappers_check_shapes(q):
    c = q.QuantCache.empty(4, 2, 16, 64, device="cpu")
    with pytest.raises(TypeError):
        c.c
    with pytest.raises(ValueError):
        q.QuantCache(c.pool, c.summary, 32, 64)
    with pytest.raises(ValueError):
        q.QuantCache(c.pool, c.summary.float(), 16, 64)
    with pytest.raises(ValueError):
        q.QuantCache(c.pool.to(torch.int8), c.summary, 16, 64)
    with pytest.raises(ValueError):
        q.QKNorm(torch.ones(64), torch.ones(2, 63)).check(4, 2, 64, -1)
    with pytest.raises(ValueError):
        q.QKNorm(torch.ones(64).half(), None).check(4, 2, 64, -1)
    q.QKNorm(torch.ones(4, 64), torch.ones(64)).check(4, 2, 64, -1)
