"""The normed append (norm, rotation, cache write in one pass) against its fp64 form."""

import numpy as np
import pytest
import torch

from oracle import quest_oracle as qo
from tests._cases import F16, F32, dev_i32, gpu_table, np_of
from tests._dense_ref import rotate, rotate_tol
from tests.test_gpu_rope_append import HALF, _bits, _inputs

pytestmark = pytest.mark.gpu

LENS, BEFORE = [1, 0, 33, 16, 5, 70], [0, 7, 15, 16, 31, 3]
EPS = 1e-5

# Of a normed element, relative: the sum of squares is a chain of 16 products, a tree over at
# most 16 lanes and the mean (21 roundings of 2^-24, halved by the root), rsqrtf (2 ulp, 4 of
# 2^-24), the products with the weight and with the element: 17 of 2^-24.
NORM_ERR = 17 * 2.0 ** -24


def _weights(seed, h, group, d, per_head):
    g = torch.Generator().manual_seed(seed)
    shape = lambda n: (n, d) if per_head else (d,)  # noqa: E731
    return tuple((1 + 0.5 * torch.randn(shape(n), generator=g)).cuda() for n in (h * group, h))


def normed(x, w):
    x = np.asarray(x, np.float64)
    return x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * np_of(w).astype(np.float64)


def close_to_form(got, x, w, pos, freq, interleaved, half_step):
    """got [n, heads, d] against norm and rotation of x; freq None: no rotation."""
    y = normed(x, w)
    if freq is None:
        tol = np.abs(y) * half_step + 2.0 ** -25
        size = np.zeros_like(y)
    else:
        flat, size = rotate(y, pos, freq, interleaved)
        tol = rotate_tol(flat, size, pos, freq, interleaved, half_step)
        y = flat
    if w is not None:
        tol = tol + NORM_ERR * (size + np.abs(y))
    err = np.abs(got.astype(np.float64) - y)
    assert np.all(err <= tol), float((err / tol).max())


def _check(seed, lens, before, *, h=2, group=2, d=128, S=16, dtype=F16, rotary=None, interleaved=False, fp8=False,
           rope=True, per_head=False, sides="qk", positions=None, pad=0, with_q=True):
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(seed, lens, before, h, group, d, S, dtype, fp8, pad)
    ind = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    inv = qs.rope_frequencies(rotary or d) if rope else None
    wq, wk = _weights(seed, h, group, d, per_head)
    norm = qs.QKNorm(wq if "q" in sides else None, wk if "k" in sides else None, EPS)
    start = [x.clone() for x in (cache.k_pool, cache.v_pool, cache.summary)]
    q_out = qs.norm_rope_append_kv(cache, gpu_table(table), q if with_q else None, k, v, dev_i32(ind), dev_i32(before),
                                   norm, group, inv_freq=inv, interleaved=interleaved,
                                   positions=None if positions is None else dev_i32(positions))
    assert qs.device_error() == 0
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, lens)] or [[]])
    turn = pos if positions is None else np.asarray(positions)
    f = np_of(inv) if rope else None
    if with_q:
        close_to_form(np_of(q_out), np_of(q), norm.q_weight, turn, f, interleaved, HALF[dtype])
    else:
        assert q_out is None
    req = np.repeat(np.arange(len(lens)), lens)
    phys = table.page_indices[table.page_indptr[req] + pos // S]
    got = np_of(cache.k_pool)[phys, :, pos % S]
    close_to_form(got, np_of(k), norm.k_weight, turn, f, interleaved, HALF[dtype])
    # everything else bit for bit from the keys as stored
    okp, ovp, osm = (np_of(x) for x in start)
    if fp8:
        okp[phys, :, pos % S], ovp[phys, :, pos % S] = got, np_of(v)
        for r in range(table.batch):
            for p in range(table.pages_of(r)):
                pp = table.page_indices[table.page_indptr[r] + p]
                if pp in phys:
                    cnt = min(S, int(table.seq_lens[r]) - p * S)
                    box = np.stack([okp[pp, :, :cnt].min(1), okp[pp, :, :cnt].max(1)], 1)
                    osm[pp] = qo.summary_to_e4m3(box)[0]
    else:
        qo.append_kv(okp, ovp, osm, table.page_indptr, table.page_indices, np.asarray(before), ind, got, np_of(v))
    for x, y in zip((cache.k_pool, cache.v_pool, cache.summary), (okp, ovp, osm)):
        assert np.array_equal(_bits(np_of(x)), _bits(y))


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (64, 16), (128, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, d, S, interleaved):
    _check(1, LENS, BEFORE, d=d, S=S, dtype=dtype, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,d,rotary", [(F16, 128, 64), (F16, 128, 16), (F16, 64, 48), (F32, 128, 112), (F32, 64, 16)])
def test_rotates_a_part(dtype, d, rotary, interleaved):
    _check(2, LENS, BEFORE, d=d, dtype=dtype, rotary=rotary, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("over", [dict(rope=False), dict(per_head=True), dict(sides="q"), dict(sides="k"),
                                  dict(with_q=False), dict(rope=False, per_head=True, with_q=False)])
def test_what_is_done(dtype, over):
    _check(3, LENS, BEFORE, h=3, d=64, dtype=dtype, **over)


@pytest.mark.parametrize("group,h,pad", [(1, 3, 0), (8, 1, 64), (4, 5, 8), (1, 40, 0)])
def test_heads_and_strides(group, h, pad):
    _check(4, LENS, BEFORE, h=h, group=group, d=64, pad=pad, per_head=True)


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32)])
def test_e4m3_summaries(d, S):
    _check(5, LENS, BEFORE, d=d, S=S, fp8=True)


def _as_they_are(x, S=16, fp8=False):
    """x [n, h, d] as keys that are neither normed nor rotated, a request each."""
    import query_aware_sparse_gb300 as qs
    n, h, d = x.shape
    cache = qs.PagedCache.empty(n, h, S, d, F16, summary_fp8=fp8)
    table = qs.PageTable(dev_i32(np.arange(n + 1)), dev_i32(np.arange(n)), dev_i32(np.ones(n)))
    k = torch.from_numpy(x).cuda()
    qs.norm_rope_append_kv(cache, table, None, k, k, dev_i32(np.arange(n + 1)), dev_i32(np.zeros(n)), qs.QKNorm(None, None), 1)
    assert np.array_equal(_bits(np_of(cache.k_pool)[:, :, 0]), _bits(x))
    return np_of(cache.summary)


@pytest.mark.parametrize("d", [64, 128])
def test_e4m3_summary_of_every_fp16_number(d):
    """Pages of one token each: the box of a number is its floor and its ceiling."""
    import query_aware_sparse_gb300 as qs
    bits = np.arange(1 << 16, dtype=np.uint16)
    bits = bits[bits & 0x7c00 != 0x7c00]
    x = bits.view(np.float16).reshape(-1, 1, d)
    got = _as_they_are(x, fp8=True)
    assert qs.device_error() == 0x10
    assert np.array_equal(got, qo.summary_to_e4m3(np.stack([x, x], 2))[0])
    small = x[(np.abs(x) <= 448).all(-1)[:, 0]]
    _as_they_are(np.ascontiguousarray(small), fp8=True)
    assert qs.device_error() == 0


def test_zeros_keep_their_order():
    """-0 below +0, in fp16 boxes as in fp32 ones."""
    for dtype in (F16, F32):
        for d, S in ((128, 16), (64, 32)):
            import query_aware_sparse_gb300 as qs
            rng = np.random.default_rng(1)
            x = np.where(rng.random((S, 2, d)) < 0.5, 0.0, -0.0).astype(np.float16 if dtype == F16 else np.float32)
            x[:3] = rng.normal(size=(3, 2, d)) * (rng.random((3, 2, d)) < 0.3)
            cache = qs.PagedCache.empty(1, 2, S, d, dtype)
            table = qs.PageTable(dev_i32([0, 1]), dev_i32([0]), dev_i32([S]))
            k = torch.from_numpy(x).cuda()
            for a, b in ((0, 5), (5, S)):
                qs.norm_rope_append_kv(cache, table, None, k[a:b], k[a:b], dev_i32([0, b - a]), dev_i32([a]),
                                       qs.QKNorm(None, None), 1)
            okp, ovp, osm = (np.zeros(t.shape, x.dtype) for t in (cache.k_pool, cache.v_pool, cache.summary))
            qo.append_kv(okp, ovp, osm, np.array([0, 1]), np.array([0]), np.zeros(1, np.int32), np.array([0, S]), x, x)
            assert np.array_equal(_bits(np_of(cache.summary)), _bits(osm))


def test_one_token_and_batches():
    _check(6, [1], [0], h=1, group=1)
    rng = np.random.default_rng(1)
    _check(7, [1] * 75, rng.integers(0, 50, 75).tolist(), h=2, group=1, d=64)
    _check(8, [10007], [5], h=1, group=1)
    _check(9, rng.integers(0, 3, 800).tolist(), rng.integers(0, 40, 800).tolist(), h=1, group=2, d=64)


@pytest.mark.parametrize("dtype,d,S", [(F16, 128, 16), (F16, 64, 32), (F16, 128, 32), (F32, 128, 16), (F32, 64, 32)])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_long_request_among_many_without_tokens(dtype, d, S, fp8):
    """Few tokens per request on average, and pages full of them all the same."""
    if dtype == F16 or not fp8:
        _check(14, [50] + [0] * 20 + [3, 1], [5] + [9] * 20 + [15, 16], d=d, S=S, dtype=dtype, fp8=fp8, interleaved=fp8)


def test_positions():
    rng = np.random.default_rng(2)
    p = rng.integers(-2 ** 31, 2 ** 31, sum(LENS))
    _check(10, LENS, BEFORE, d=64, dtype=F32, positions=p, interleaved=True)


def test_in_place_padding_and_bad_pages():
    """q_out = q; rows behind the last request stay; without a page the queries
    are treated all the same."""
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(11, [20, 3], [0, 30], 2, 2, 64, 16, F16)
    wq, wk = _weights(11, 2, 2, 64, False)
    norm, inv = qs.QKNorm(wq, wk, EPS), qs.rope_frequencies(64)
    ind, before = dev_i32([0, 20, 22]), dev_i32([0, 30])
    t = gpu_table(table)
    want = qs.norm_rope_append_kv(cache, t, q, k, v, ind, before, norm, 2, inv_freq=inv,
                                  q_out=torch.full((23, 4, 64), 3.0, dtype=F16, device="cuda"))
    assert (want[22] == 3).all() and not (want[21] == 3).all()
    dense = q.contiguous()
    last = dense[22].clone()
    qs.norm_rope_append_kv(cache, t, dense, k, v, ind, before, norm, 2, inv_freq=inv, q_out=dense)
    assert torch.equal(dense[:22], want[:22]) and torch.equal(dense[22], last)
    assert qs.device_error() == 0
    pools = [x.clone() for x in (cache.k_pool, cache.v_pool, cache.summary)]
    t.page_indices[0] = -1
    t.page_indices[1] = cache.n_phys
    got = qs.norm_rope_append_kv(cache, t, q, k, v, dev_i32([0, 20, 20]), before, norm, 2, inv_freq=inv)
    assert qs.device_error() == 1 and torch.equal(got[:20], want[:20])
    for x, y in zip(pools, (cache.k_pool, cache.v_pool, cache.summary)):
        assert np.array_equal(_bits(np_of(x)), _bits(np_of(y)))


def test_small_and_large_rows():
    """Rows of zeros, of the smallest numbers (eps decides) and of the largest."""
    import query_aware_sparse_gb300 as qs
    for dtype, big in ((F16, 65504.0), (F32, 1e17)):
        table, cache, q, k, v = _inputs(12, [8], [0], 1, 1, 64, 16, dtype)
        scale = torch.tensor([0.0, 2.0 ** -24, 1e-5, 1e-2, 1.0, 1e2, big / 8, big], device="cuda")[:, None, None]
        k = (k.float() / k.float().abs().amax(-1, keepdim=True) * scale).to(dtype)
        wq, wk = _weights(12, 1, 1, 64, False)
        qs.norm_rope_append_kv(cache, gpu_table(table), None, k, v, dev_i32([0, 8]), dev_i32([0]),
                               qs.QKNorm(wq, wk, EPS), 1, inv_freq=qs.rope_frequencies(64))
        got = np_of(cache.k_pool)[table.page_indices[0], :, :8].transpose(1, 0, 2)
        close_to_form(got, np_of(k), wk, np.arange(8), np_of(qs.rope_frequencies(64)), False, HALF[dtype])


def test_same_bits_on_another_stream_and_in_a_graph():
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(13, [40, 9], [3, 30], 2, 2, 128, 16, F16)
    wq, wk = _weights(13, 2, 2, 128, True)
    norm, inv, t = qs.QKNorm(wq, wk, EPS), qs.rope_frequencies(128), gpu_table(table)
    ind, before = dev_i32([0, 40, 49]), dev_i32([3, 30])
    call = lambda **kw: qs.norm_rope_append_kv(cache, t, q, k, v, ind, before, norm, 2, inv_freq=inv, **kw)  # noqa: E731
    want, pool = call(), cache.k_pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(q_out=out)
    cache.k_pool.zero_()
    g.replay()
    held = ~pool.isnan()
    assert torch.equal(out, want)
    new = np.concatenate([np.arange(3, 43), np.arange(30, 39)])
    rows = np.repeat([0, 1], [40, 9])
    phys = torch.as_tensor(table.page_indices[table.page_indptr[rows] + new // 16]).long().cuda()
    slot = torch.as_tensor(new % 16).long().cuda()
    assert held[phys, :, slot].all() and torch.equal(cache.k_pool[phys, :, slot], pool[phys, :, slot])
