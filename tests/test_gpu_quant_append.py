"""Appends into the E4M3 cache, byte for byte, and its read-back."""

import numpy as np
import pytest
import torch

import workloads as wl
from oracle import quest_oracle as qo
from tests._cases import F16, dev_i32, gpu_table, np_of
from tests._quant_ref import gpu_quant, k_at, quant_case, quantise, stored, v_at
from tests.test_gpu_norm_append import EPS, _weights
from tests.test_gpu_rope_append import _bits

pytestmark = pytest.mark.gpu

LENS, BEFORE = [1, 0, 33, 16, 5, 70], [0, 7, 15, 16, 31, 3]
FP8_RANGE = 0x10


def _summary_of(box, fp8):
    return qo.summary_to_e4m3(box)[0] if fp8 else box


def _decode_summary(s):
    if s.dtype != np.uint8:
        return s
    return torch.from_numpy(np.ascontiguousarray(s)).view(torch.float8_e4m3fn).half().numpy()


def _check(seed, lens, before, *, h=2, group=2, d=128, S=16, fp8=False, rope=False, norm=False, interleaved=False,
           rotary=None, pad=0, k=None, v=None, with_q=None, error=0):
    import query_aware_sparse_gb300 as qs
    table = wl.make_page_table(np.asarray(lens) + np.asarray(before), S, seed=seed, permute=True, spare_pages=3)
    g = torch.Generator().manual_seed(seed)
    n, hq = int(np.sum(lens)), h * group
    row = torch.randn((n, (hq + 2 * h) * d + pad), generator=g).half().cuda()
    q = row[:, :hq * d].view(n, hq, d)
    k = row[:, hq * d:(hq + h) * d].view(n, h, d) if k is None else k
    v = row[:, (hq + h) * d:(hq + 2 * h) * d].view(n, h, d) if v is None else v
    rng = np.random.default_rng(seed)
    rec = rng.integers(0, 256, (table.n_phys, h, 2 * S * (d + 1)), dtype=np.uint8)
    old = np.sort(rng.normal(size=(table.n_phys, h, 2, d)), axis=2).astype(np.float16) * 3
    sm = _summary_of(old, fp8)
    cache = qs.QuantCache(torch.from_numpy(rec.copy()).cuda(), torch.from_numpy(sm.copy()).cuda(), S, d)
    ind = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    inv = qs.rope_frequencies(rotary or d) if rope else None
    qk = qs.QKNorm(*_weights(seed, h, group, d, False), EPS) if norm else None
    with_q = rope or norm if with_q is None else with_q
    args = (gpu_table(table), q if with_q else None, k, v, dev_i32(ind), dev_i32(before))
    q_out = qs.quant_append_kv(cache, *args, group, inv_freq=inv, norm=qk, interleaved=interleaved)
    assert qs.device_error() == error
    # the keys as the fp16 append keeps them
    keys = np_of(k)
    pos = np.concatenate([np.arange(b, b + m) for b, m in zip(before, lens)] or [[]]).astype(int)
    req = np.repeat(np.arange(len(lens)), lens)
    phys = table.page_indices[table.page_indptr[req] + pos // S]
    if rope or norm:
        plain = qs.PagedCache.empty(table.n_phys, h, S, d, F16)
        want_q = qs.norm_rope_append_kv(plain, *args, qk or qs.QKNorm(None, None), group, inv_freq=inv,
                                        interleaved=interleaved)
        qs.device_error()
        assert (q_out is None) == (not with_q) and (not with_q or torch.equal(q_out, want_q))
        keys = np_of(plain.k_pool)[phys, :, pos % S]
    kc, ke, _ = quantise(keys)
    vc, ve, _ = quantise(np_of(v))
    for i in range(n):
        p, t = phys[i], pos[i] % S
        rec[p][:, k_at(S, d)[t]] = kc[i]
        rec[p][:, v_at(S, d)[t]] = vc[i]
        rec[p][:, 2 * S * d + t] = ke[i] + 127
        rec[p][:, 2 * S * d + S + t] = ve[i] + 127
    got = np_of(cache.pool)
    # a zero has two codes: its sign is the input's in both
    assert np.array_equal(got, rec), np.argwhere(got != rec)[:5]
    kept = stored(kc, ke)
    for p in np.unique(phys):
        mine = phys == p
        box = np.stack([kept[mine].min(0), kept[mine].max(0)], 1)
        if not (pos[mine] % S == 0).any():
            was = _decode_summary(sm[p])
            box = np.stack([np.minimum(box[:, 0], was[:, 0]), np.maximum(box[:, 1], was[:, 1])], 1)
        sm[p] = _summary_of(box, fp8)
    # the order -0 < +0 is the fp16 summary's own affair (test_gpu_append.py)
    assert np.array_equal(_decode_summary(np_of(cache.summary)), _decode_summary(sm))
    return cache, table


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (64, 16), (128, 32)])
@pytest.mark.parametrize("fp8", [False, True])
def test_append(d, S, fp8):
    _check(1, LENS, BEFORE, d=d, S=S, fp8=fp8)


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rope,norm,part", [(True, False, 1), (True, True, 1), (False, True, 1), (True, True, 2)])
def test_append_of_treated_keys(d, S, interleaved, rope, norm, part):
    _check(2, LENS, BEFORE, d=d, S=S, rope=rope, norm=norm, interleaved=interleaved, rotary=d // part)


@pytest.mark.parametrize("group,h,pad", [(1, 3, 0), (8, 1, 64), (4, 5, 8), (1, 40, 0)])
def test_heads_and_strides(group, h, pad):
    _check(3, LENS, BEFORE, h=h, group=group, d=64, pad=pad, rope=True)


def test_one_token_and_batches():
    _check(4, [1], [0], h=1, group=1)
    _check(5, [1], [4095], h=4, group=8, S=32, norm=True)
    rng = np.random.default_rng(1)
    _check(6, [1] * 75, rng.integers(0, 50, 75).tolist(), d=64, rope=True)
    _check(7, [3007], [5], h=1, group=1)
    _check(8, rng.integers(0, 3, 400).tolist(), rng.integers(0, 40, 400).tolist(), h=1, d=64)
    _check(9, LENS, BEFORE, rope=True, with_q=False)


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (64, 16), (128, 32)])
def test_a_long_request_among_many_without_tokens(d, S):
    _check(17, [50] + [0] * 20 + [3, 1], [5] + [9] * 20 + [15, 16], d=d, S=S, norm=True, rope=True)


@pytest.mark.parametrize("d", [64, 128])
def test_every_magnitude(d):
    """Rows whose largest element runs through the fp16 numbers around each
    power of two and the borders 448 * 2^e, with elements down to zero."""
    tops = []
    for e in range(-24, 16):
        for m in (1.0, 1 + 2.0 ** -10, 1.5, 1.75 - 2.0 ** -10, 1.75, 1.75 + 2.0 ** -10, 2 - 2.0 ** -10):
            if m * 2.0 ** e <= 57344:
                tops.append(m * 2.0 ** e)
    tops = np.asarray(tops + [0.0, 57344.0]).astype(np.float16)
    n = len(tops)
    rng = np.random.default_rng(3)
    x = rng.normal(size=(n, 2, d)) * 2.0 ** rng.integers(-14, 1, (n, 2, d))
    x = np.clip(x / np.abs(x).max(-1, keepdims=True), -1, 1) * tops[:, None, None].astype(np.float64)
    x = np.clip(x.astype(np.float16), -tops[:, None, None], tops[:, None, None])
    x[:, :, 5] = tops[:, None]
    x[:, 1] *= np.float16(-1)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    _check(10, [n], [0], d=d, k=dev(x), v=dev(x[::-1]))


def test_ties_round_to_even():
    """Numbers half way between two codes."""
    c = torch.arange(0, 0x7e, dtype=torch.uint8)
    lo, hi = (t.view(torch.float8_e4m3fn).float() for t in (c, c + 1))
    mid = ((lo + hi) / 2).half()
    assert torch.equal(mid.float(), (lo + hi) / 2)
    x = torch.zeros((2, 1, 128), dtype=F16)
    x[0, 0, :126], x[1, 0, :126] = mid, -mid
    x[:, 0, 126] = 448.0
    _check(11, [2], [3], h=1, k=x.cuda(), v=x.flip(0).contiguous().cuda())


def test_what_cannot_be_kept_is_reported():
    x = torch.randn((20, 2, 128), generator=torch.Generator().manual_seed(4)).half()
    for at, value in (((3, 0, 7), 65504.0), ((4, 1, 0), float("inf")), ((5, 0, 127), -float("inf")),
                      ((6, 1, 64), float("nan")), ((19, 1, 3), -57376.0)):
        x[at] = value
    fine = torch.randn((20, 2, 128), generator=torch.Generator().manual_seed(5)).half()
    _check(12, [20], [9], k=x.cuda(), v=fine.cuda(), error=FP8_RANGE)
    _check(13, [20], [9], k=fine.cuda(), v=x.cuda(), error=FP8_RANGE)
    _check(16, [20], [9], k=(fine * 300).cuda(), v=fine.cuda(), fp8=True, error=FP8_RANGE)   # beyond the summary's range
    fine[0, 0, 0] = 57344.0
    _check(14, [20], [9], k=fine.cuda(), v=fine.cuda())


def test_bad_pages_padding_and_repeats():
    import query_aware_sparse_gb300 as qs
    cache, table = _check(15, [40, 9], [3, 30], rope=True)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn((52, 2, 128), generator=g).half().cuda() for _ in range(2))
    q = torch.randn((52, 4, 128), generator=g).half().cuda()
    inv, t = qs.rope_frequencies(128), gpu_table(table)
    q_out = torch.full_like(q, 3)
    before = [x.clone() for x in (cache.pool, cache.summary)]
    t.page_indices[:3] = torch.tensor([-1, cache.n_phys, 1 << 30], dtype=torch.int32)
    qs.quant_append_kv(cache, t, q, k, v, dev_i32([0, 40, 40]), dev_i32([3, 30]), 2, inv_freq=inv, q_out=q_out)
    assert qs.device_error() == 1
    assert torch.equal(cache.pool, before[0]) and torch.equal(cache.summary, before[1])
    assert (q_out[40:] == 3).all() and not (q_out[39] == 3).all()
    # beyond the table
    qs.quant_append_kv(cache, gpu_table(table), None, k, v, dev_i32([0, 0, 52]), dev_i32([3, 30]), 2, inv_freq=inv)
    assert qs.device_error() == 2
    # a graph's replay and another stream write the same bytes
    t = gpu_table(table)
    cache.pool.copy_(before[0])
    args = (t, q, k, v, dev_i32([0, 40, 49]), dev_i32([3, 30]), 2)
    out = qs.quant_append_kv(cache, *args, inv_freq=inv)
    want = cache.pool.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        qs.quant_append_kv(cache, *args, inv_freq=inv, q_out=q_out)
    cache.pool.copy_(before[0])
    gr.replay()
    side = torch.cuda.Stream()
    assert torch.equal(q_out[:49], out[:49]) and qs.device_error() == 0
    new = cache.pool.clone()
    side.wait_stream(torch.cuda.current_stream())
    qs.quant_append_kv(cache, *args, inv_freq=inv, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(new, cache.pool)
    assert torch.equal(new, want)


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (64, 16), (128, 32)])
@pytest.mark.parametrize("indexed", [False, True])
def test_read_back(d, S, indexed):
    """Every token's number, other slots as they were."""
    import query_aware_sparse_gb300 as qs
    lens = [1, 0, 15, 16, 17, 33, 643, 0, 100]
    case = quant_case(21, lens, h_kv=3, d=d, S=S, reserve_tokens=40)
    cache, t = gpu_quant(case), case["table"]
    n_dst = t.nnz + 4
    dst = qs.PagedCache.empty(n_dst, 3, S, d, F16)
    for x in (dst.k_pool, dst.v_pool, dst.summary):
        x.fill_(-7.0)
    at = np.random.default_rng(2).permutation(n_dst)[:t.nnz] if indexed else np.arange(t.nnz)
    qs.quant_read_kv(cache, gpu_table(t), dst, dst_indices=dev_i32(at) if indexed else None)
    assert qs.device_error() == 0 and (dst.summary == -7).all()
    for pool, src in ((dst.k_pool, case["k_pool"]), (dst.v_pool, case["v_pool"])):
        want = np.full((n_dst, 3, S, d), -7.0, np.float16)
        rows = np_of(src)[t.page_indices]
        want[at] = np.where(np.isnan(rows), np.float16(-7), rows)
        # reserved pages hold no token
        for r, n in enumerate(lens):
            for p in range(-(-n // S), int(t.page_indptr[r + 1] - t.page_indptr[r])):
                want[at[t.page_indptr[r] + p]] = -7.0
        assert np.array_equal(np_of(pool), want)


def test_read_back_bad_pages_and_large_batch():
    import query_aware_sparse_gb300 as qs
    rng = np.random.default_rng(5)
    case = quant_case(22, rng.integers(0, 40, 1100).tolist(), h_kv=1, d=64, S=16)
    cache, t = gpu_quant(case), case["table"]
    dst = qs.PagedCache.empty(t.nnz, 1, 16, 64, F16)
    dst.k_pool.fill_(-7.0)
    idx = np.arange(t.nnz)
    idx[5], idx[9] = -1, t.nnz
    bad = t.page_indices.copy()
    bad[[20, 31]] = [-3, t.n_phys]
    table = gpu_table(t)
    table.page_indices.copy_(dev_i32(bad))
    qs.quant_read_kv(cache, table, dst, dst_indices=dev_i32(idx))
    assert qs.device_error() == 1
    want = np_of(case["k_pool"])[t.page_indices]
    want = np.where(np.isnan(want), np.float16(-7), want)
    want[[5, 9, 20, 31]] = -7.0
    assert np.array_equal(np_of(dst.k_pool), want)
    longer = t.seq_lens.copy()
    longer[-1] = 100000
    qs.quant_read_kv(cache, gpu_table(t, seq_lens=longer), dst)
    assert qs.device_error() == 2


def test_views_are_the_documented_layout():
    case = quant_case(23, [70, 9], h_kv=2, d=64, S=32)
    cache = gpu_quant(case)
    kc = cache.k_codes.permute(0, 1, 3, 2, 4).reshape(-1, 2, 32, 64)
    vc = cache.v_codes.permute(0, 1, 2, 7, 5, 8, 3, 4, 6).reshape(-1, 2, 32, 64)
    held = torch.from_numpy(~case["empty_slots"]).cuda()
    for codes, scales, pool in ((kc, cache.k_scales, case["k_pool"]), (vc, cache.v_scales, case["v_pool"])):
        x = codes.float() * scales.float()[..., None]
        assert torch.equal(x[held], pool.cuda().float()[held])


def test_far_pages():
    """Records beyond 2^32 bytes of the pool."""
    import query_aware_sparse_gb300 as qs
    h, S, d = 8, 16, 128
    n_phys = (1 << 32) // (h * qs.quant_page_bytes(S, d)) + 40
    cache = qs.QuantCache.empty(n_phys, h, S, d)
    ids = dev_i32([n_phys - 1, 3, n_phys - 30])
    table = qs.PageTable(dev_i32([0, 3]), ids, dev_i32([45]))
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((45, h, d), generator=g, device="cuda").half() for _ in range(2))
    qs.quant_append_kv(cache, table, None, k, v, dev_i32([0, 45]), dev_i32([0]), 1)
    dst = qs.PagedCache.empty(3, h, S, d, F16)
    qs.quant_read_kv(cache, table, dst)
    q = torch.randn((1, h, d), generator=g, device="cuda").half()
    sel = torch.arange(3, dtype=torch.int32, device="cuda").expand(1, h, 3).contiguous()
    phys = ids.expand(1, h, 3).contiguous()
    same = qs.PageTable(dev_i32([0, 3]), dev_i32([0, 1, 2]), dev_i32([45]))
    want, _ = qs.dense_decode_attn(dst, same, q, 1)
    for out, _ in (qs.quant_dense_decode_attn(cache, table, q, 1),
                   qs.quant_sparse_decode_attn(cache, table, q, 1, sel, phys, 3)):
        assert (out - want).abs().max() <= 2.0 ** -18
    assert qs.device_error() == 0
    kk = dst.k_pool.transpose(1, 2).reshape(-1, h, d)[:45]
    c, e, _ = quantise(np_of(k))
    assert np.array_equal(_bits(np_of(kk)), _bits(stored(c, e)))
