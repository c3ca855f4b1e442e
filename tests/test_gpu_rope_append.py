"""The rotating append against its fp64 form, and a prompt and decode steps
through append, prompt attention, dense decode and the fused sparse step."""

import numpy as np
import pytest
import torch

import workloads as wl
from oracle import quest_oracle as qo
from tests._cases import F16, F32, attn_close, dev_i32, gpu_table, np_of
from tests._dense_ref import attention, check_attention, rotate, rotate_tol

pytestmark = pytest.mark.gpu

HALF = {F16: 2.0 ** -11, F32: 2.0 ** -24}


def _bits(a):
    a = np.ascontiguousarray(a)
    return a.view({1: np.uint8, 2: np.uint16, 4: np.uint32}[a.itemsize])


def _inputs(seed, lens, before, h, group, d, S, dtype, fp8=False, pad=0):
    """A pool whose requests already hold before[r] tokens, and the parts of a
    fused projection with `pad` extra elements per row."""
    import query_aware_sparse_gb300 as qs
    table = wl.make_page_table(np.asarray(lens) + np.asarray(before), S, seed=seed, permute=True, spare_pages=3)
    g = torch.Generator().manual_seed(seed)
    n, hq = int(np.sum(lens)), h * group
    row = torch.randn((n, (hq + 2 * h) * d + pad), generator=g).to(dtype).cuda()
    q = row[:, :hq * d].view(n, hq, d)
    k = row[:, hq * d:(hq + h) * d].view(n, h, d)
    v = row[:, (hq + h) * d:(hq + 2 * h) * d].view(n, h, d)
    cache = qs.PagedCache.empty(table.n_phys, h, S, d, dtype, summary_fp8=fp8)
    cache.k_pool.fill_(float("nan"))
    cache.v_pool.fill_(float("nan"))
    cache.summary.fill_(0 if fp8 else float("nan"))
    old = torch.randn((int(np.sum(before)), h, d), generator=g).to(dtype).cuda()
    zero = np.zeros(len(lens), np.int32)
    t0 = gpu_table(table, seq_lens=np.asarray(before, np.int32))
    qs.append_kv(cache, t0, old, old, dev_i32(np.concatenate([[0], np.cumsum(before)])), dev_i32(zero))
    return table, cache, q, k, v


def _check(seed, lens, before, *, h=2, group=2, d=128, S=16, dtype=F16, rotary=None, interleaved=False,
           fp8=False, base=10000.0, positions=None, pad=0, with_q=True):
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(seed, lens, before, h, group, d, S, dtype, fp8, pad)
    ind = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    inv = qs.rope_frequencies(rotary or d, base)
    start = [x.clone() for x in (cache.k_pool, cache.v_pool, cache.summary)]
    q_out = qs.rope_append_kv(cache, gpu_table(table), q if with_q else None, k, v, dev_i32(ind), dev_i32(before),
                              inv, group, interleaved=interleaved,
                              positions=None if positions is None else dev_i32(positions))
    assert qs.device_error() == 0
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, lens)] or [[]])
    turn = pos if positions is None else np.asarray(positions)
    f = np_of(inv)
    if with_q:
        y, size = rotate(np_of(q), turn, f, interleaved)
        err = np.abs(np_of(q_out).astype(np.float64) - y)
        assert np.all(err <= rotate_tol(y, size, turn, f, interleaved, HALF[dtype])), err.max()
        tail = np_of(q)[..., (rotary or d):]
        assert np.array_equal(_bits(np_of(q_out)[..., (rotary or d):]), _bits(tail))
    else:
        assert q_out is None
    # the keys as stored, and everything else bit for bit from them
    req = np.repeat(np.arange(len(lens)), lens)
    phys = table.page_indices[table.page_indptr[req] + pos // S]
    got = np_of(cache.k_pool)[phys, :, pos % S]
    y, size = rotate(np_of(k), turn, f, interleaved)
    err = np.abs(got.astype(np.float64) - y)
    assert np.all(err <= rotate_tol(y, size, turn, f, interleaved, HALF[dtype])), err.max()
    okp, ovp = np_of(start[0]), np_of(start[1])
    if fp8:
        osm = np_of(start[2])
        full = np.full(osm.shape, np.nan, np.float16)
        okp[phys, :, pos % S], ovp[phys, :, pos % S] = got, np_of(v)
        for pp in np.unique(phys):
            r, p = [(r, p) for r in range(table.batch) for p in range(table.pages_of(r))
                    if table.page_indices[table.page_indptr[r] + p] == pp][0]
            cnt = min(S, int(table.seq_lens[r]) - p * S)
            full[pp, :, 0], full[pp, :, 1] = okp[pp, :, :cnt].min(1), okp[pp, :, :cnt].max(1)
        codes, _ = qo.summary_to_e4m3(full[np.unique(phys)])
        osm[np.unique(phys)] = codes
    else:
        osm = np_of(start[2])
        qo.append_kv(okp, ovp, osm, table.page_indptr, table.page_indices, np.asarray(before), ind, got, np_of(v))
    assert np.array_equal(_bits(np_of(cache.k_pool)), _bits(okp))
    assert np.array_equal(_bits(np_of(cache.v_pool)), _bits(ovp))
    assert np.array_equal(_bits(np_of(cache.summary)), _bits(osm))


LENS, BEFORE = [1, 0, 33, 16, 5, 70], [0, 7, 15, 16, 31, 3]


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (64, 16), (128, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, d, S, interleaved):
    _check(1, LENS, BEFORE, d=d, S=S, dtype=dtype, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,d,rotary", [(F16, 128, 64), (F16, 128, 16), (F16, 64, 48), (F32, 128, 112),
                                            (F32, 64, 16), (F16, 128, 112)])
def test_append_rotates_a_part(dtype, d, rotary, interleaved):
    _check(2, LENS, BEFORE, d=d, dtype=dtype, rotary=rotary, interleaved=interleaved)


@pytest.mark.parametrize("group,h,pad", [(1, 3, 0), (8, 1, 64), (4, 5, 8), (1, 40, 0)])
def test_append_heads_and_strides(group, h, pad):
    _check(3, LENS, BEFORE, h=h, group=group, d=64, pad=pad)


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32)])
def test_append_e4m3(d, S):
    _check(4, LENS, BEFORE, d=d, S=S, fp8=True)


def test_append_one_token_and_decode_batch():
    _check(5, [1], [0], h=1, group=1)
    _check(6, [1], [4095], h=4, group=8)
    rng = np.random.default_rng(1)
    _check(7, [1] * 75, rng.integers(0, 50, 75).tolist(), h=2, group=1, d=64)


def test_append_many_pages_of_few_heads():
    """Enough pages to fill the device several times over, from one request and
    from hundreds."""
    _check(17, [10007], [5], h=1, group=1)
    rng = np.random.default_rng(4)
    _check(18, rng.integers(0, 3, 800).tolist(), rng.integers(0, 40, 800).tolist(), h=1, group=2, d=64)


def test_append_without_queries():
    _check(8, LENS, BEFORE, with_q=False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_positions(interleaved):
    """Positions of the caller's, as far as 2^31 - 1 and below zero."""
    rng = np.random.default_rng(2)
    n = sum(LENS)
    p = rng.integers(-2 ** 31, 2 ** 31, n)
    p[:3] = [2 ** 31 - 1, -2 ** 31, 0]
    _check(9, LENS, BEFORE, d=64, dtype=F32, positions=p, interleaved=interleaved)
    _check(10, LENS, BEFORE, d=64, positions=np.full(n, 1000003), base=500000.0, interleaved=interleaved)


def test_append_in_place_and_padding():
    """q_out = q, and rows behind the last request left as they were."""
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(11, [20, 3], [0, 30], 2, 2, 64, 16, F16)
    inv = qs.rope_frequencies(64)
    ind = dev_i32([0, 20, 22])                       # the last row belongs to nobody
    want = qs.rope_append_kv(cache, gpu_table(table), q, k, v, ind, dev_i32([0, 30]), inv, 2,
                             q_out=torch.full((23, 4, 64), 3.0, dtype=F16, device="cuda"))
    assert (want[22] == 3).all() and not (want[21] == 3).all()
    dense = q.contiguous()
    last = dense[22].clone()
    pools = [x.clone() for x in (cache.k_pool, cache.v_pool, cache.summary)]
    qs.rope_append_kv(cache, gpu_table(table), dense, k, v, ind, dev_i32([0, 30]), inv, 2, q_out=dense)
    assert torch.equal(dense[:22], want[:22]) and torch.equal(dense[22], last)
    for x, y in zip(pools, (cache.k_pool, cache.v_pool, cache.summary)):
        assert np.array_equal(_bits(np_of(x)), _bits(np_of(y)))       # folding the same keys again
    assert qs.device_error() == 0


def test_append_bad_pages_are_reported_and_queries_rotated():
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(12, [40, 20], [0, 0], 2, 2, 64, 16, F16)
    inv = qs.rope_frequencies(64)
    t = gpu_table(table)
    ind, before = dev_i32([0, 40, 60]), dev_i32([0, 0])
    want = qs.rope_append_kv(cache, t, q, k, v, ind, before, inv, 2)
    kp = cache.k_pool.clone()
    table.page_indices[1] = table.n_phys
    cache.k_pool.fill_(5.0)
    got = qs.rope_append_kv(cache, gpu_table(table), q, k, v, ind, before, inv, 2)
    assert qs.device_error() == 1 and torch.equal(got, want)
    bad = wl.make_page_table([40, 20], 16, seed=12, permute=True, spare_pages=3).page_indices[1]
    assert (cache.k_pool[int(bad)] == 5).all()
    table.page_indices[1] = bad
    got = qs.rope_append_kv(cache, gpu_table(table), q, k, v, ind, dev_i32([0, 25]), inv, 2)
    assert qs.device_error() == 2 and torch.equal(got[:40], want[:40])
    assert torch.equal(cache.k_pool[int(bad)], kp[int(bad)])


def test_append_flags_keys_beyond_e4m3():
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(13, [20], [0], 2, 2, 64, 16, F16, fp8=True)
    k[7, 1, 5] = 1000.0
    qs.rope_append_kv(cache, gpu_table(table), None, k, v, dev_i32([0, 20]), dev_i32([0]),
                      qs.rope_frequencies(64), 2)
    assert qs.device_error() == 16


def test_append_replays():
    import query_aware_sparse_gb300 as qs
    table, cache, q, k, v = _inputs(14, [30, 1], [0, 17], 2, 4, 128, 16, F16)
    args = (gpu_table(table), q, k, v, dev_i32([0, 30, 31]), dev_i32([0, 17]), qs.rope_frequencies(128), 4)
    out = torch.empty((31, 8, 128), dtype=F16, device="cuda")
    qs.rope_append_kv(cache, *args, q_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.rope_append_kv(cache, *args, q_out=out)
    q.mul_(-2)
    g.replay()
    want = qs.rope_append_kv(cache, *args)
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype,group,d,S", [(F16, 4, 128, 16), (F32, 2, 64, 32), (F16, 1, 64, 16)])
def test_prompt_then_decode_through_all_operators(dtype, group, d, S):
    """Two requests' prompts in two chunks each, then decode steps: rotate and
    append, prompt attention, dense decode; a fused sparse step whose budget
    covers every page agrees with dense decode."""
    import query_aware_sparse_gb300 as qs
    h, total, chunks = 2, [150, 61], [[100, 16], [45, 40]]
    hq = h * group
    table = wl.make_page_table(total, S, seed=5, permute=True, spare_pages=2)
    g = torch.Generator().manual_seed(77)
    tok = [[torch.randn((n, x, d), generator=g).to(dtype) for x in (hq, h, h)] for n in total]
    inv = qs.rope_frequencies(d)
    cache = qs.PagedCache.empty(table.n_phys, h, S, d, dtype)
    cache.k_pool.fill_(float("nan"))
    cache.v_pool.fill_(float("nan"))
    done, half = np.zeros(2, np.int64), (2.0 ** -11 if dtype == F16 else 0.0)
    steps = chunks + [[1, 1]] * 5
    for step in steps:
        part = [torch.cat([tok[r][i][done[r]:done[r] + step[r]] for r in range(2)]).cuda() for i in range(3)]
        ind = np.concatenate([[0], np.cumsum(step)]).astype(np.int32)
        after = gpu_table(table, seq_lens=(done + step).astype(np.int32))
        q = qs.rope_append_kv(cache, after, *part, dev_i32(ind), dev_i32(done), inv, group)
        done = done + step
        # the reference reads the rotated keys and queries as stored
        ref = attention(np_of(q), np_of(cache.k_pool), np_of(cache.v_pool), table.page_indptr, table.page_indices,
                        done, ind, group)
        if max(step) > 1:
            out, lse = qs.prefill_attn(cache, after, q, group, dev_i32(ind))
            check_attention(np_of(out), np_of(lse), ref, half, half, int(done.max()))
            continue
        out, lse = qs.dense_decode_attn(cache, after, q, group)
        check_attention(np_of(out), np_of(lse), ref, 0.0, 0.0, int(done.max()))
        again, _ = qs.prefill_attn(cache, after, q, group, dev_i32(ind))
        check_attention(np_of(again), np_of(lse), ref, half, half, int(done.max()))
        sparse = qs.DecodeStep(cache, after, group, max(table.pages_of(r) for r in range(2)))
        so, sl = sparse(cache, after, q)
        assert attn_close(np_of(so), np_of(out))[0].all()
    assert qs.device_error() == 0
    # against the rotation of the tokens themselves, end to end
    for r in range(2):
        y, size = rotate(np_of(tok[r][1][:done[r]]), np.arange(done[r]), np_of(inv), False)
        ids = table.page_indices[table.page_indptr[r] + np.arange(done[r]) // S]
        got = np_of(cache.k_pool)[ids, :, np.arange(done[r]) % S].astype(np.float64)
        tol = rotate_tol(y, size, np.arange(done[r]), np_of(inv), False, HALF[dtype])
        assert np.all(np.abs(got - y) <= tol)
