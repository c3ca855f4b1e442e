"""Dense decode and prompt attention against their fp64 form."""

import numpy as np
import pytest
import torch

from tests._cases import F16, F32, dev_i32, gpu_cache, gpu_table, np_of, random_case
from tests._dense_ref import attention, check_attention

pytestmark = pytest.mark.gpu

# One rounding, relative: half a step of the type (fp16 2^-11). The softmax
# weights are rounded to fp16 in prompt attention with fp16 keys; dense decode
# keeps them to 2^-22 and better.
HALF16 = 2.0 ** -11


def _mods(case, rows, seed, kinds):
    """Keyword arguments for the reference and a ScoreMods of the same values."""
    import query_aware_sparse_gb300 as qs
    rng = np.random.default_rng(seed)
    hq, lens = case["h_kv"] * case["group"], case["table"].seq_lens
    kw = {}
    if "cap" in kinds:
        kw["softcap"] = 3.0
    if "window" in kinds:
        kw["window"] = 37
    if "alibi" in kinds:
        kw["slopes"] = (2.0 ** -rng.uniform(0, 8, hq)).astype(np.float32)
    if "doc" in kinds:
        ends = [np.arange(L - n, L) for L, n in zip(lens, rows)]
        kw["doc_starts"] = np.concatenate([np.maximum(0, e // 50 * 50) for e in ends]).astype(np.int32)
        if len(kw["doc_starts"]) > 2:
            kw["doc_starts"][2] = 1 << 30          # this row sees nothing
            kw["doc_starts"][0] = -5
    if "prefix" in kinds:
        kw["prefix_lens"] = rng.integers(0, 90, len(lens)).astype(np.int32)
    names = {"slopes": "alibi_slopes"}
    dev = {names.get(k, k): torch.as_tensor(v, device="cuda") if isinstance(v, np.ndarray) else v
           for k, v in kw.items()}
    return kw, qs.ScoreMods(**dev)


def _reference(case, q, q_indptr, table=None, seq_lens=None, **kw):
    t = case["table"] if table is None else table
    return attention(np_of(q), np_of(case["k_pool"]), np_of(case["v_pool"]), t.page_indptr,
                     t.page_indices, t.seq_lens if seq_lens is None else seq_lens, q_indptr,
                     case["group"], **kw)


def _decode(case, kinds=(), seed=0, **over):
    import query_aware_sparse_gb300 as qs
    B = case["table"].batch
    kw, mods = _mods(case, [1] * B, seed, kinds)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    out, lse = qs.dense_decode_attn(cache, table, case["q"].cuda(), case["group"],
                                    mods=mods if kinds else None, **over)
    assert qs.device_error() == 0
    ref = _reference(case, case["q"], np.arange(B + 1), **kw)
    check_attention(np_of(out), np_of(lse), ref, 0.0, 0.0, int(case["table"].seq_lens.max()))
    return out, lse


def _rows_case(seed, lens, rows, dtype=F16, **shape):
    """random_case with rows[r] query rows per request."""
    case = random_case(seed, lens, dtype=dtype, **shape)
    g = torch.Generator().manual_seed(seed + 99)
    case["q"] = torch.randn((sum(rows), case["h_kv"] * case["group"], case["d"]), generator=g).to(dtype)
    case["rows"] = rows
    case["q_indptr"] = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return case


def _prefill(case, kinds=(), seed=0, **over):
    import query_aware_sparse_gb300 as qs
    kw, mods = _mods(case, case["rows"], seed, kinds)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    out, lse = qs.prefill_attn(cache, table, case["q"].cuda(), case["group"], dev_i32(case["q_indptr"]),
                               mods=mods if kinds else None, **over)
    assert qs.device_error() == 0
    assert out.dtype == case["dtype"]
    ref = _reference(case, case["q"], case["q_indptr"], **kw)
    half = HALF16 if case["dtype"] == F16 else 0.0
    check_attention(np_of(out), np_of(lse), ref, half, half, int(case["table"].seq_lens.max()))
    return out, lse


LENS = [1, 0, 15, 16, 17, 31, 33, 100, 643]


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (128, 32), (64, 16)])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_decode(dtype, d, S, group):
    _decode(random_case(10 + group, LENS, h_kv=3, group=group, d=d, S=S, dtype=dtype))


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("kinds", ["cap", "alibi", "window", "doc", "prefix", "cap window alibi doc"])
def test_decode_mods(dtype, kinds):
    _decode(random_case(31, LENS, h_kv=2, group=4, d=64, S=16, dtype=dtype), kinds.split(), seed=5)


@pytest.mark.parametrize("dtype,group,h", [(F16, 4, 2), (F16, 1, 3), (F32, 2, 1), (F16, 8, 1)])
def test_decode_long_ragged(dtype, group, h):
    _decode(random_case(41, [20000, 3, 4097, 0, 9000], h_kv=h, group=group, d=128, S=16, dtype=dtype))


def test_decode_single_request_every_length():
    for n in (1, 2, 15, 16, 17, 48, 127, 128, 129, 500):
        _decode(random_case(n, [n], h_kv=1, group=1, d=64, S=16, dtype=F16))


def test_decode_large_batch():
    rng = np.random.default_rng(3)
    _decode(random_case(51, rng.integers(0, 60, 1100).tolist(), h_kv=1, group=2, d=64, S=16, dtype=F16))


def test_decode_large_scores():
    """Logits of several hundred, rising along the cache: the running maximum
    moves all the time and nothing overflows."""
    case = random_case(61, [3000, 700], h_kv=2, group=2, d=64, S=16, dtype=F16)
    case["q"] = (case["q"] * 0 + 8).half()
    k = case["k_pool"]
    t = case["table"]
    for r, L in enumerate(t.seq_lens):
        for p in range(-(-int(L) // 16)):
            k[t.page_indices[t.page_indptr[r] + p]] = ((p - 90) * 0.03)
    _decode(case)


def test_decode_reserved_pages_and_scale():
    case = random_case(71, [40, 0, 333], h_kv=2, group=2, d=64, S=16, dtype=F16, reserve_tokens=100)
    import query_aware_sparse_gb300 as qs
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    out, lse = qs.dense_decode_attn(cache, table, case["q"].cuda(), 2, sm_scale=0.31)
    ref = _reference(case, case["q"], np.arange(4), scale=float(np.float32(0.31)))
    check_attention(np_of(out), np_of(lse), ref, 0.0, 0.0, 333)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_decode_bad_pages_are_skipped_and_reported(dtype):
    import query_aware_sparse_gb300 as qs
    case = random_case(81, [100, 200, 64], h_kv=2, group=2, d=64, S=16, dtype=dtype)
    t = case["table"]
    t.page_indices[t.page_indptr[1] + 3] = t.n_phys            # just outside
    t.page_indices[t.page_indptr[1] + 12] = -1                 # the tail page
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(t)
    out, lse = qs.dense_decode_attn(cache, table, case["q"].cuda(), 2)
    assert qs.device_error() == 1
    ref = _reference(case, case["q"], np.arange(4))
    check_attention(np_of(out), np_of(lse), ref, 0.0, 0.0, 200)
    # more tokens than the table holds: the rest is skipped
    t.page_indices[:] = np.arange(t.nnz)
    longer = np.asarray([100, 208, 9999], np.int32)
    out, lse = qs.dense_decode_attn(cache, gpu_table(t, seq_lens=longer), case["q"].cuda(), 2)
    assert qs.device_error() == 2
    full = np.nan_to_num(np_of(case["k_pool"])), np.nan_to_num(np_of(case["v_pool"]))
    cache = qs.PagedCache(torch.as_tensor(full[0]).cuda(), torch.as_tensor(full[1]).cuda(), cache.summary)
    out, lse = qs.dense_decode_attn(cache, gpu_table(t, seq_lens=longer), case["q"].cuda(), 2)
    assert qs.device_error() == 2
    ref = attention(np_of(case["q"]), *full, t.page_indptr, t.page_indices, longer, np.arange(4), 2)
    check_attention(np_of(out), np_of(lse), ref, 0.0, 0.0, 208)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d,S,group", [(128, 16, 1), (64, 32, 2), (128, 32, 4), (64, 16, 8), (128, 16, 8)])
def test_prefill(dtype, d, S, group):
    lens = [1, 0, 17, 129, 300, 260, 64]
    rows = [1, 0, 17, 129, 40, 1, 33]
    _prefill(_rows_case(20 + group, lens, rows, h_kv=2, group=group, d=d, S=S, dtype=dtype))


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("kinds", ["cap", "alibi", "window", "doc", "prefix", "cap window alibi doc prefix"])
def test_prefill_mods(dtype, kinds):
    lens, rows = [200, 77, 1, 310], [200, 20, 1, 140]
    for d, S, group in ((64, 16, 4), (128, 32, 1)):
        _prefill(_rows_case(33, lens, rows, h_kv=2, group=group, d=d, S=S, dtype=dtype), kinds.split(), seed=6)


@pytest.mark.parametrize("rows", [1, 2, 3, 16, 31, 33])
@pytest.mark.parametrize("group", [1, 4])
def test_prefill_few_rows_of_a_long_cache(rows, group):
    _prefill(_rows_case(43, [6000, 2500], [rows, min(rows, 5)], h_kv=2, group=group, d=128, S=16))


@pytest.mark.parametrize("group,d", [(1, 128), (8, 64), (2, 128)])
def test_prefill_long_prompt(group, d):
    n = 1200 // group + 7
    _prefill(_rows_case(44, [n + 600, 37], [n, 37], h_kv=1, group=group, d=d, S=16))


@pytest.mark.parametrize("rows,window", [(520, 0), (2100, 0), (520, 4500)])
def test_prefill_of_a_cache_beyond_l2_share(rows, window):
    """Keys of more KV heads than stay in L2 together: heads run in groups, and
    rows are checked here and there."""
    import query_aware_sparse_gb300 as qs
    h, d, S, L = 9, 128, 16, 17003
    g = torch.Generator(device="cuda").manual_seed(rows)
    pages = -(-L // S)
    kp = torch.randn((pages, h, S, d), generator=g, device="cuda").half()
    vp = torch.randn((pages, h, S, d), generator=g, device="cuda").half()
    cache = qs.PagedCache(kp, vp, torch.zeros((pages, h, 2, d), dtype=F16, device="cuda"))
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = qs.PageTable(dev_i32([0, pages]), ids, dev_i32([L]))
    q = torch.randn((rows, h, d), generator=g, device="cuda").half()
    out, lse = qs.prefill_attn(cache, table, q, 1, dev_i32([0, rows]), mods=qs.ScoreMods(window=window))
    k = kp[ids.long()].transpose(1, 2).reshape(-1, h, d)[:L].double()
    v = vp[ids.long()].transpose(1, 2).reshape(-1, h, d)[:L].double()
    for i in (0, 1, 127, 128, 255, 256, 511, rows - 2, rows - 1):
        p = L - rows + i
        lo = max(0, p - window + 1) if window else 0
        x = torch.einsum("hd,jhd->hj", q[i].double(), k[lo:p + 1]) / d ** 0.5
        z = torch.logsumexp(x, 1)
        w = torch.exp(x - z[:, None])
        o = torch.einsum("hj,jhd->hd", w, v[lo:p + 1])
        mean = torch.einsum("hj,jhd->hd", w, v[lo:p + 1].abs())
        # weights and output each rounded to fp16; logits to 132 roundings of sum |q k| / sqrt(d)
        # (about 7: 5.6e-5, twice in a weight), 1127 roundings of 2^-24 in a row's sums (6.7e-5)
        assert ((out[i].double() - o).abs() <= mean * (HALF16 + 2e-4) + o.abs() * HALF16 + 1e-7).all(), i
        assert ((lse[i].double() - z).abs() <= 1e-4).all(), i
    assert qs.device_error() == 0


def test_prefill_large_scores():
    case = _rows_case(62, [900], [300], h_kv=1, group=2, d=64, S=16)
    case["q"] = (case["q"] * 0 + 8).half()
    t = case["table"]
    for p in range(-(-900 // 16)):
        case["k_pool"][t.page_indices[p]] = ((p - 30) * 0.1)
    _prefill(case)
    case["k_pool"] *= -1
    _prefill(case)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_prefill_more_rows_than_tokens(dtype):
    """A request with more rows than tokens: its first rows stand before the
    cache and see nothing."""
    _prefill(_rows_case(45, [5, 40], [12, 40], h_kv=2, group=2, d=64, S=16, dtype=dtype))


@pytest.mark.parametrize("dtype", [F16, F32])
def test_prefill_leaves_rows_behind_the_last_request(dtype):
    import query_aware_sparse_gb300 as qs
    case = _rows_case(46, [60, 30], [60, 11], h_kv=2, group=2, d=64, S=16, dtype=dtype)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    q = torch.cat([case["q"], torch.full((9, 4, 64), float("nan"), dtype=dtype)])
    out = torch.full((80, 4, 64), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((80, 4), 7.0, device="cuda")
    qs.prefill_attn(cache, table, q.cuda(), 2, dev_i32(case["q_indptr"]), out=out, lse=lse)
    assert qs.device_error() == 0
    assert (out[71:] == 7).all() and (lse[71:] == 7).all()
    half = HALF16 if dtype == F16 else 0.0
    check_attention(np_of(out[:71]), np_of(lse[:71]), _reference(case, case["q"], case["q_indptr"]),
                    half, half, 60)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_prefill_bad_pages_are_skipped_and_reported(dtype):
    import query_aware_sparse_gb300 as qs
    case = _rows_case(82, [300, 200], [150, 200], h_kv=2, group=2, d=64, S=16, dtype=dtype)
    t = case["table"]
    t.page_indices[t.page_indptr[0] + 3] = -7
    t.page_indices[t.page_indptr[0] + 18] = t.n_phys + 100      # the tail page
    t.page_indices[t.page_indptr[1]] = 1 << 30
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(t)
    out, lse = qs.prefill_attn(cache, table, case["q"].cuda(), 2, dev_i32(case["q_indptr"]))
    assert qs.device_error() == 1
    half = HALF16 if dtype == F16 else 0.0
    check_attention(np_of(out), np_of(lse), _reference(case, case["q"], case["q_indptr"]), half, half, 300)


def _both(case, cache, table, ws_d, ws_p, out, stream=None):
    import query_aware_sparse_gb300 as qs
    B = case["table"].batch
    qs.dense_decode_attn(cache, table, case["qd"], case["group"], out=out[0], lse=out[1], workspace=ws_d,
                         stream=stream)
    qs.prefill_attn(cache, table, case["qp"], case["group"], case["ind"], out=out[2], lse=out[3],
                    workspace=ws_p, stream=stream)


def _setup(seed=91):
    import query_aware_sparse_gb300 as qs
    lens, rows = [3000, 17, 900], [3, 17, 200]
    case = _rows_case(seed, lens, rows, h_kv=2, group=2, d=128, S=16)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    case["qd"], case["qp"], case["ind"] = case["q"][:3].cuda().contiguous(), case["q"].cuda(), dev_i32(case["q_indptr"])
    ws_d = torch.zeros(max(16, qs.dense_decode_workspace_size(3, table.nnz, 2, 2, 128, 16, F16)), dtype=torch.uint8, device="cuda")
    ws_p = torch.zeros(max(16, qs.prefill_workspace_size(3, 220, table.nnz, 2, 2, 128, 16, F16)), dtype=torch.uint8, device="cuda")
    new = lambda: (torch.empty((3, 4, 128), device="cuda"), torch.empty((3, 4), device="cuda"),
                   torch.empty((220, 4, 128), dtype=F16, device="cuda"), torch.empty((220, 4), device="cuda"))
    return case, cache, table, ws_d, ws_p, new


def test_attention_repeats_bit_for_bit_and_replays():
    """The same call gives the same bits: run again in its workspace, on
    another stream, captured and replayed with new queries."""
    case, cache, table, ws_d, ws_p, new = _setup()
    a, b, c = new(), new(), new()
    _both(case, cache, table, ws_d, ws_p, a)
    for _ in range(5):
        _both(case, cache, table, ws_d, ws_p, b)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _both(case, cache, table, ws_d, ws_p, c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _both(case, cache, table, ws_d, ws_p, c)
    qd, qp = case["qd"].clone(), case["qp"].clone()
    case["qd"].neg_()
    case["qp"].neg_()
    g.replay()
    _both(case, cache, table, ws_d, ws_p, b)
    assert all(torch.equal(x, y) for x, y in zip(b, c))
    assert not torch.equal(a[0], b[0]) and not torch.equal(a[2], b[2])
    case["qd"].copy_(qd)
    case["qp"].copy_(qp)
    g.replay()
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(a, c))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace."""
    case, cache, table, ws_d, ws_p, new = _setup(95)
    want, got = new(), [new(), new()]
    _both(case, cache, table, ws_d, ws_p, want)
    torch.cuda.synchronize()
    spaces = [(ws_d, ws_p), (torch.empty_like(ws_d), torch.empty_like(ws_p))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for s, w, g in zip(streams, spaces, got):
            _both(case, cache, table, *w, g, stream=s)
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(want, g))


def test_results_of_another_stream():
    """A call on a side stream does not write into memory that the current stream
    gave back while its work on it was still to come."""
    import query_aware_sparse_gb300 as q
    torch.manual_seed(11)
    cache = q.PagedCache(*(torch.randn(64, 2, 16, 128, device="cuda", dtype=torch.float16) for _ in range(2)),
                         torch.empty(64, 2, 2, 128, device="cuda", dtype=torch.float16))
    i32 = dict(dtype=torch.int32, device="cuda")
    table = q.PageTable(torch.tensor([0, 64], **i32), torch.arange(64, **i32), torch.tensor([1000], **i32))
    x = torch.randn(300, 8, 128, device="cuda", dtype=torch.float16)
    rows = torch.tensor([0, 300], **i32)
    kv, before = x[:, :2].contiguous(), torch.tensor([700], **i32)
    freq, side = q.rope_frequencies(128), torch.cuda.Stream()

    def calls(stream):
        # (the append comes last: it changes what the others read)
        yield lambda: q.dense_decode_attn(cache, table, x[:1], 4, stream=stream)
        yield lambda: q.prefill_attn(cache, table, x, 4, rows, stream=stream)
        yield lambda: (q.rope_append_kv(cache, table, x, kv, kv, rows, before, freq, 4, stream=stream),)
    for plain, other in zip(calls(None), calls(side)):
        want = plain()
        want = [w.clone() for w in want]
        other()                                        # (loads what the call needs)
        torch.cuda.synchronize()
        junk = [torch.empty_like(w) for w in want]
        torch.cuda._sleep(20_000_000)
        for j in junk:
            j.fill_(7.0)
        del junk, j
        got = other()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_requests_that_share_pages():
    """The same physical pages as the prefix of two requests, and twice in one."""
    import query_aware_sparse_gb300 as qs
    case = _rows_case(96, [100, 80, 64], [40, 9, 64], h_kv=2, group=2, d=64, S=16)
    t = case["table"]
    t.page_indices[t.page_indptr[1]:t.page_indptr[1] + 4] = t.page_indices[:4]
    t.page_indices[t.page_indptr[2] + 1] = t.page_indices[t.page_indptr[2]]
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(t)
    out, lse = qs.prefill_attn(cache, table, case["q"].cuda(), 2, dev_i32(case["q_indptr"]))
    check_attention(np_of(out), np_of(lse), _reference(case, case["q"], case["q_indptr"]), HALF16, HALF16, 100)
    out, lse = qs.dense_decode_attn(cache, table, case["q"][:3].cuda().contiguous(), 2)
    check_attention(np_of(out), np_of(lse), _reference(case, case["q"][:3], np.arange(4)), 0.0, 0.0, 100)
    assert qs.device_error() == 0


@pytest.mark.parametrize("dtype", [F16, F32])
def test_nothing_to_see(dtype):
    """Requests without a token, and rows that belong to no request."""
    import query_aware_sparse_gb300 as qs
    case = random_case(97, [0, 0, 0], h_kv=2, group=2, d=64, S=16, dtype=dtype)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    assert table.nnz == 0
    q = case["q"].cuda()
    out, lse = qs.dense_decode_attn(cache, table, q, 2)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = qs.prefill_attn(cache, table, q, 2, dev_i32([0, 1, 1, 3]))
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = torch.full_like(out, 5), torch.full_like(lse, 5)
    qs.prefill_attn(cache, table, q, 2, dev_i32([0, 0, 0, 0]), out=out, lse=lse)
    assert (out == 5).all() and (lse == 5).all() and qs.device_error() == 0


@pytest.mark.parametrize("dtype", [F16, F32])
def test_padded_batch(dtype):
    """A few requests among hundreds of empty ones."""
    lens = [0] * 700
    for i, n in ((0, 37), (150, 1), (151, 900), (420, 64), (699, 33)):
        lens[i] = n
    _decode(random_case(98, lens, h_kv=2, group=2, d=64, S=16, dtype=dtype))
    rows = [min(n, 40) for n in lens]
    _prefill(_rows_case(99, lens, rows, h_kv=1, group=2, d=64, S=16, dtype=dtype))


@pytest.mark.parametrize("dtype", [F16, F32])
def test_prefill_large_batch(dtype):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 50, 300).tolist()
    _prefill(_rows_case(100, lens, [min(n, int(k)) for n, k in zip(lens, rng.integers(0, 9, 300))],
                        h_kv=1, group=4, d=64, S=16, dtype=dtype))


@pytest.mark.parametrize("dtype", [F16, F32])
def test_window_of_one_and_many_heads(dtype):
    """Each row sees itself: out = v, lse = its own logit."""
    import query_aware_sparse_gb300 as qs
    case = _rows_case(101, [70, 5], [70, 5], h_kv=40, group=8, d=64, S=32, dtype=dtype)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    out, lse = qs.prefill_attn(cache, table, case["q"].cuda(), 8, dev_i32(case["q_indptr"]),
                               mods=qs.ScoreMods(window=1))
    v = case["v_tok"].repeat_interleave(8, dim=1)
    half = 2.0 ** -11 if dtype == F16 else 2.0 ** -22
    assert (np.abs(np_of(out).astype(np.float64) - np_of(v)) <= 2 * half * np.abs(np_of(v)) + 1e-7).all()
    last = case["q"][[69, 74]].cuda()
    out, lse = qs.dense_decode_attn(cache, table, last, 8, mods=qs.ScoreMods(window=1))
    assert (np.abs(np_of(out) - np_of(v[[69, 74]]).astype(np.float64)) <= 2.0 ** -20 * np.abs(np_of(v[[69, 74]])) + 1e-7).all()


def test_without_lse():
    """lse may be NULL in the C calls."""
    import ctypes
    import query_aware_sparse_gb300 as qs
    case, cache, table, ws_d, ws_p, new = _setup(102)
    want, out = new(), new()
    _both(case, cache, table, ws_d, ws_p, want)
    by, s = ctypes.byref, torch.cuda.current_stream().cuda_stream
    L, F = qs.lib(), ctypes.c_float(0.0)
    assert L.quest_dense_decode_attn(by(cache.c), by(table.c), case["qd"].data_ptr(), 2, None, out[0].data_ptr(), None,
                                     F, ws_d.data_ptr(), ws_d.numel(), s) == 0
    assert L.quest_prefill_attn(by(cache.c), by(table.c), case["qp"].data_ptr(), 2, case["ind"].data_ptr(), 220, None,
                                out[2].data_ptr(), None, F, ws_p.data_ptr(), ws_p.numel(), s) == 0
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])


def test_workspace_serves_smaller_calls_after_larger_ones():
    import query_aware_sparse_gb300 as qs
    case, cache, table, ws_d, ws_p, new = _setup(92)
    a, b = new(), new()
    _both(case, cache, table, ws_d, ws_p, a)
    small = random_case(93, [40, 0, 700], h_kv=2, group=2, d=128, S=16)
    sc, st = gpu_cache(small["k_pool"], small["v_pool"], small["summary"]), gpu_table(small["table"])
    out, lse = qs.dense_decode_attn(sc, st, small["q"].cuda(), 2, workspace=ws_d)
    check_attention(np_of(out), np_of(lse), _reference(small, small["q"], np.arange(4)), 0.0, 0.0, 700)
    _both(case, cache, table, ws_d, ws_p, b)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert qs.device_error() == 0


@pytest.mark.parametrize("group,d,rows", [(2, 128, [3, 17, 200]), (4, 64, [1, 17, 300])])
def test_attention_of_buffers_on_16_byte_boundaries(group, d, rows):
    """Queries, outputs and workspaces that start 16 bytes into an allocation."""
    import query_aware_sparse_gb300 as qs
    lens = [3000, 17, 900]
    case = _rows_case(94, lens, rows, h_kv=2, group=group, d=d, S=16)
    hq, n = 2 * group, sum(rows)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])

    def off(shape, dtype):
        size = int(np.prod(shape))
        t = torch.zeros(size + 64, dtype=dtype, device="cuda")
        step = 16 // t.element_size()
        return t[step:step + size].view(shape)
    q = off((n, hq, d), F16).copy_(case["q"])
    args = (3, table.nnz, 2, group, d, 16, F16)
    out, lse = off((n, hq, d), F16), off((n, hq), torch.float32)
    qs.prefill_attn(cache, table, q, group, dev_i32(case["q_indptr"]), out=out, lse=lse,
                    workspace=off((qs.prefill_workspace_size(3, n, *args[1:]),), torch.uint8))
    check_attention(np_of(out), np_of(lse), _reference(case, case["q"], case["q_indptr"]), HALF16, HALF16, 3000)
    out, lse = off((3, hq, d), torch.float32), off((3, hq), torch.float32)
    qs.dense_decode_attn(cache, table, off((3, hq, d), F16).copy_(case["q"][:3]), group, out=out, lse=lse,
                         workspace=off((qs.dense_decode_workspace_size(*args),), torch.uint8))
    check_attention(np_of(out), np_of(lse), _reference(case, case["q"][:3], np.arange(4)), 0.0, 0.0, 3000)
    assert qs.device_error() == 0


def test_attention_of_far_pages():
    """Pages whose offset in the pool passes 2^31 elements and 2^32 bytes."""
    import query_aware_sparse_gb300 as qs
    h, S, d = 8, 32, 128
    n_phys = (1 << 31) // (h * S * d) + 40
    kp = torch.zeros((n_phys, h, S, d), dtype=F16, device="cuda")
    vp = torch.zeros_like(kp)
    cache = qs.PagedCache(kp, vp, torch.zeros((n_phys, h, 2, d), dtype=F16, device="cuda"))
    L = 300
    pages = n_phys - 1 - np.arange(10)
    g = torch.Generator().manual_seed(7)
    ids = torch.as_tensor(pages.copy(), device="cuda")
    kp[ids] = torch.randn((10, h, S, d), generator=g).half().cuda()
    vp[ids] = torch.randn((10, h, S, d), generator=g).half().cuda()
    table = qs.PageTable(dev_i32([0, 10]), dev_i32(pages), dev_i32([L]))
    q = torch.randn((40, h, d), generator=g).half()
    small = [np_of(x[ids]) for x in (kp, vp)]
    out, lse = qs.dense_decode_attn(cache, table, q[39:].cuda(), 1)
    ref = attention(np_of(q[39:]), *small, [0, 10], np.arange(10), [L], [0, 1], 1)
    check_attention(np_of(out), np_of(lse), ref, 0.0, 0.0, L)
    out, lse = qs.prefill_attn(cache, table, q.cuda(), 1, dev_i32([0, 40]))
    ref = attention(np_of(q), *small, [0, 10], np.arange(10), [L], [0, 40], 1)
    check_attention(np_of(out), np_of(lse), ref, HALF16, HALF16, L)
    assert qs.device_error() == 0
