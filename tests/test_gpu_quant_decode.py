"""Sparse and dense decode over the E4M3 cache against their fp64 forms on the
stored numbers, and the cache through a model's steps."""

import numpy as np
import pytest
import torch

from oracle import quest_oracle as qo
from tests._cases import F16, dev_i32, gpu_table, np_of
from tests._dense_ref import attention, check_attention
from tests._quant_ref import fill, gpu_quant, quant_case, requantise
from tests.test_gpu_dense import _mods
from tests.test_gpu_dense_fault import _recovers

pytestmark = pytest.mark.gpu

LENS = [1, 0, 15, 16, 17, 31, 33, 100, 643]


def _reference(case, table=None, seq_lens=None, **kw):
    t = case["table"] if table is None else table
    return attention(np_of(case["q"]), np_of(case["k_pool"]), np_of(case["v_pool"]), t.page_indptr, t.page_indices,
                     t.seq_lens if seq_lens is None else seq_lens, np.arange(t.batch + 1), case["group"], **kw)


def _dense(case, kinds=(), seed=0, **over):
    import query_aware_sparse_gb300 as qs
    kw, mods = _mods(case, [1] * case["table"].batch, seed, kinds)
    out, lse = qs.quant_dense_decode_attn(gpu_quant(case), gpu_table(case["table"]), case["q"].cuda(), case["group"],
                                          mods=mods if kinds else None, **over)
    assert qs.device_error() == 0
    check_attention(np_of(out), np_of(lse), _reference(case, **kw), 0.0, 0.0, int(case["table"].seq_lens.max()))
    return out, lse


def _lists(case, k, seed=0, drop=0.0):
    """Random distinct pages of each (request, head), in increasing order, -1 behind them."""
    t, h = case["table"], case["h_kv"]
    rng = np.random.default_rng(seed)
    sel = np.full((t.batch, h, k), -1, np.int32)
    phys = sel.copy()
    for r in range(t.batch):
        P = -(-int(t.seq_lens[r]) // case["S"])
        for g in range(h):
            pick = np.sort(rng.permutation(P)[:k])
            sel[r, g, :len(pick)] = pick
            phys[r, g, :len(pick)] = t.page_indices[t.page_indptr[r] + pick]
            if drop:
                sel[r, g, rng.random(k) < drop] = -1
    return sel, phys


def _sparse_reference(case, sel, scale=None):
    """fp64 form over the listed pages: each (request, head) as a request of its own."""
    t, h, G, S = case["table"], case["h_kv"], case["group"], case["S"]
    out, lse = [], []
    parts = []
    for r in range(t.batch):
        for g in range(h):
            pages = np.sort(sel[r, g][sel[r, g] >= 0])
            L = int(t.seq_lens[r])
            n = sum(min(S, L - p * S) for p in pages)
            ids = t.page_indices[t.page_indptr[r] + pages] if len(pages) else np.zeros(0, np.int32)
            kp, vp = np_of(case["k_pool"])[:, g:g + 1], np_of(case["v_pool"])[:, g:g + 1]
            parts.append(attention(np_of(case["q"])[r:r + 1, g * G:(g + 1) * G], kp, vp, [0, len(ids)], ids, [n], [0, 1],
                                   G, scale=scale))
    return {k: np.concatenate([p[k][0] for p in parts]).reshape((t.batch, h * G) + parts[0][k].shape[2:]) for k in parts[0]}


def _sparse(case, k, seed=0, drop=0.0, **over):
    import query_aware_sparse_gb300 as qs
    sel, phys = _lists(case, k, seed, drop)
    out, lse = qs.quant_sparse_decode_attn(gpu_quant(case), gpu_table(case["table"]), case["q"].cuda(), case["group"],
                                           dev_i32(sel), dev_i32(phys), k, **over)
    assert qs.device_error() == 0
    check_attention(np_of(out), np_of(lse), _sparse_reference(case, sel), 0.0, 0.0, k * case["S"])
    return out, lse


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (128, 32), (64, 16)])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_dense(d, S, group):
    _dense(quant_case(10 + group, LENS, h_kv=3, group=group, d=d, S=S))


@pytest.mark.parametrize("kinds", ["cap", "alibi", "window", "doc", "prefix", "cap window alibi doc"])
@pytest.mark.parametrize("d,S", [(64, 16), (128, 32)])
def test_dense_mods(kinds, d, S):
    _dense(quant_case(31, LENS, h_kv=2, group=4, d=d, S=S), kinds.split(), seed=5)


@pytest.mark.parametrize("group,h", [(4, 2), (1, 3), (8, 1)])
def test_dense_long_ragged(group, h):
    _dense(quant_case(41, [20000, 3, 4097, 0, 9000], h_kv=h, group=group, d=128, S=16))


def test_dense_every_length():
    for n in (1, 2, 15, 16, 17, 31, 32, 33, 48, 127, 128, 129, 500):
        for S in (16, 32):
            _dense(quant_case(n, [n], h_kv=1, group=1, d=64, S=S))


def test_dense_large_batch():
    rng = np.random.default_rng(3)
    _dense(quant_case(51, rng.integers(0, 60, 1100).tolist(), h_kv=1, group=2, d=64, S=16))


@pytest.mark.parametrize("d,S", [(128, 16), (64, 32), (128, 32), (64, 16)])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_sparse(d, S, group):
    case = quant_case(60 + group, LENS, h_kv=3, group=group, d=d, S=S)
    _sparse(case, 7, seed=group)
    _sparse(case, 50, seed=group, drop=0.3)


@pytest.mark.parametrize("k", [1, 2, 3, 31, 32, 33, 300])
def test_sparse_budgets(k):
    _sparse(quant_case(70, [5000, 17, 0, 900], h_kv=2, group=4, d=128, S=16), k, seed=k)


def test_sparse_large_batch():
    rng = np.random.default_rng(4)
    _sparse(quant_case(71, rng.integers(0, 200, 300).tolist(), h_kv=2, group=1, d=64, S=16), 5)


def test_scales_of_every_size():
    """Tokens whose keys and values differ by many powers of two."""
    import query_aware_sparse_gb300 as qs
    from tests._cases import random_case
    case = random_case(72, [300, 77], h_kv=2, group=2, d=128, S=16)
    rng = np.random.default_rng(5)
    f = 2.0 ** rng.integers(-12, 4, case["k_pool"].shape[:3])[..., None]
    case["k_pool"] = (case["k_pool"].double() * torch.from_numpy(f)).half()
    f = 2.0 ** rng.integers(-20, 13, case["v_pool"].shape[:3])[..., None]
    case["v_pool"] = (case["v_pool"].double() * torch.from_numpy(f)).half()
    requantise(case)
    # a weight is kept to 2^-25 where the largest is 2^6 or more: 2^-31 of the sum for each key,
    # which counts where one token's values are far larger than the others'. check_attention's
    # relative term is 2^-18 at least.
    def apart(ref, n):
        ref["aw"] = ref["aw"] + n * 2.0 ** -31 / 2.0 ** -18 * ref["vmax"][..., None]
        return ref
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    out, lse = qs.quant_dense_decode_attn(cache, t, q, 2)
    check_attention(np_of(out), np_of(lse), apart(_reference(case), 300), 0.0, 0.0, 300)
    sel, phys = _lists(case, 9, 0)
    out, lse = qs.quant_sparse_decode_attn(cache, t, q, 2, dev_i32(sel), dev_i32(phys), 9)
    check_attention(np_of(out), np_of(lse), apart(_sparse_reference(case, sel), 144), 0.0, 0.0, 144)
    assert qs.device_error() == 0


@pytest.mark.parametrize("d,S,group", [(64, 16, 2), (64, 32, 8), (128, 32, 8), (128, 32, 4), (64, 32, 1)])
def test_large_scores(d, S, group):
    """Logits of several hundred, rising token by token: the running maximum
    moves all the time, inside a page too, and nothing overflows."""
    from tests._cases import random_case
    case = random_case(61, [3000, 700], h_kv=2, group=group, d=d, S=S)
    case["q"] = (case["q"] * 0 + 8).half()
    t = case["table"]
    for r, L in enumerate(t.seq_lens):
        for p in range(-(-int(L) // S)):
            x = case["k_pool"][t.page_indices[t.page_indptr[r] + p]]
            rise = (torch.arange(S)[:, None] + p * S - 1440) * (0.12 / 64)
            x[~x.isnan()] = rise.half().expand_as(x)[~x.isnan()]
    requantise(case)
    _dense(case)
    _sparse(case, 40)


@pytest.mark.parametrize("d,S,group", [(128, 32, 8), (64, 32, 8), (128, 16, 8), (64, 16, 1), (64, 32, 4)])
def test_equal_runs(d, S, group):
    """Tables and lists that are too long for a cluster per unit, with masks."""
    case = quant_case(330 + S + group, [24000, 31, 0, 9000], h_kv=1, group=group, d=d, S=S)
    _dense(case)
    _dense(case, ["cap", "alibi", "doc"], seed=3)
    _sparse(case, 700, seed=1, drop=0.1)


def test_bad_pages_are_skipped_and_reported():
    import query_aware_sparse_gb300 as qs
    case = quant_case(81, [100, 200, 64], h_kv=2, group=2, d=64, S=16, garbage=0)
    t, q = case["table"], case["q"].cuda()
    cache = gpu_quant(case)
    sel, phys = _lists(case, 6, 1)
    keep = sel.copy()
    phys[0, 1, 2], phys[1, 0, 5] = t.n_phys, -1                # outside the pool
    keep[0, 1, 2] = keep[1, 0, 5] = -1
    out, lse = qs.quant_sparse_decode_attn(cache, gpu_table(t), q, 2, dev_i32(sel), dev_i32(phys), 6)
    assert qs.device_error() == 1
    check_attention(np_of(out), np_of(lse), _sparse_reference(case, keep), 0.0, 0.0, 96)
    sel, phys = _lists(case, 6, 1)
    keep = sel.copy()
    sel[2, 0, 5], phys[2, 0, 5] = 4, 0                          # no token there
    sel[2, 1, 5], phys[2, 1, 5] = 0x7fffffff, 0
    out, lse = qs.quant_sparse_decode_attn(cache, gpu_table(t), q, 2, dev_i32(sel), dev_i32(phys), 6)
    assert qs.device_error() == 4
    check_attention(np_of(out), np_of(lse), _sparse_reference(case, keep), 0.0, 0.0, 96)
    t.page_indices[t.page_indptr[1] + 3] = t.n_phys
    t.page_indices[t.page_indptr[1] + 12] = -1
    out, lse = qs.quant_dense_decode_attn(cache, gpu_table(t), q, 2)
    assert qs.device_error() == 1
    check_attention(np_of(out), np_of(lse), _reference(case), 0.0, 0.0, 200)
    t.page_indices[:] = np.arange(t.nnz)
    longer = np.asarray([100, 208, 9999], np.int32)
    qs.quant_dense_decode_attn(cache, gpu_table(t, seq_lens=longer), q, 2)
    assert qs.device_error() == 2


def test_nothing_to_see():
    import query_aware_sparse_gb300 as qs
    case = quant_case(82, [0, 50, 0], h_kv=2, group=2, d=64, S=16)
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    none = torch.full((3, 2, 4), -1, dtype=torch.int32, device="cuda")
    out, lse = qs.quant_sparse_decode_attn(cache, t, q, 2, none, none, 4)
    assert (out == 0).all() and lse.isneginf().all()
    docs = torch.full((3,), 1 << 30, dtype=torch.int32, device="cuda")
    out, lse = qs.quant_dense_decode_attn(cache, t, q, 2, mods=qs.ScoreMods(doc_starts=docs))
    assert (out == 0).all() and lse.isneginf().all() and qs.device_error() == 0


def test_bytes_without_a_token_change_nothing():
    import query_aware_sparse_gb300 as qs
    for d, S in ((128, 16), (64, 32)):
        case = quant_case(83, [1, 37, 200, 17], h_kv=2, group=4, d=d, S=S, garbage=0)
        t, q = gpu_table(case["table"]), case["q"].cuda()
        sel, phys = (dev_i32(x) for x in _lists(case, 5, 2))
        got = []
        for byte in (0, 0xff, 0x7f, 0x80, 0x01):
            fill(case["records"], case["empty_slots"], byte, S, d)
            cache = gpu_quant(case)
            got.append(qs.quant_dense_decode_attn(cache, t, q, 4) + qs.quant_sparse_decode_attn(cache, t, q, 4, sel, phys, 5) +
                       qs.quant_dense_decode_attn(cache, t, q, 4, mods=qs.ScoreMods(softcap=2.0, window=20)))
        for other in got[1:]:
            assert all(torch.equal(x, y) for x, y in zip(got[0], other))


def _calls(seed=91):
    import query_aware_sparse_gb300 as qs
    case = quant_case(seed, [3000, 17, 900], h_kv=2, group=2, d=128, S=16)
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    sel, phys = (dev_i32(x) for x in _lists(case, 20, 3))
    n = qs.quant_decode_workspace_size(3, 2, 2, 128, 16)
    new = lambda: (torch.empty((3, 4, 128), device="cuda"), torch.empty((3, 4), device="cuda"),  # noqa: E731
                   torch.empty((3, 4, 128), device="cuda"), torch.empty((3, 4), device="cuda"),
                   torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda"))

    def both(o, stream=None):
        qs.quant_dense_decode_attn(cache, t, q, 2, out=o[0], lse=o[1], workspace=o[4], stream=stream)
        qs.quant_sparse_decode_attn(cache, t, q, 2, sel, phys, 20, out=o[2], lse=o[3], workspace=o[4], stream=stream)
    return q, new, both


def test_repeats_bit_for_bit_and_replays():
    q, new, both = _calls()
    a, b, c = new(), new(), new()
    same = lambda x, y: all(torch.equal(u, v) for u, v in zip(x[:4], y[:4]))  # noqa: E731
    both(a)
    for _ in range(5):
        both(b)
        assert same(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(a, c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(c)
    old = q.clone()
    q.neg_()
    g.replay()
    both(b)
    assert same(b, c) and not torch.equal(a[0], b[0]) and not torch.equal(a[2], b[2])
    q.copy_(old)
    g.replay()
    g.replay()
    assert same(a, c)


def test_two_calls_at_once():
    q, new, both = _calls(95)
    want = new()
    both(want)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [new(), new()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, o in zip(streams, outs):
            both(o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(want[:4], o[:4]))


def test_one_workspace_for_calls_of_all_sizes():
    """Large and small calls, lists and tables, in any order: what one leaves in
    the workspace is nothing to the next."""
    import query_aware_sparse_gb300 as qs
    rng = np.random.default_rng(8)
    n = max(qs.quant_decode_workspace_size(300, 3, 8, d, 16) for d in (64, 128))
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    calls = []
    for i, (lens, h, G, d, S) in enumerate([([9000, 5], 2, 8, 128, 16), ([40], 1, 1, 64, 32),
                                            (rng.integers(0, 300, 300).tolist(), 3, 2, 64, 16), ([20000], 1, 8, 64, 16),
                                            ([7000, 0, 7000], 3, 4, 128, 32)]):
        case = quant_case(300 + i, lens, h_kv=h, group=G, d=d, S=S)
        sel, phys = (dev_i32(x) for x in _lists(case, 30, i))
        c, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
        calls.append(lambda c=c, t=t, q=q, G=G, **kw: qs.quant_dense_decode_attn(c, t, q, G, **kw))
        calls.append(lambda c=c, t=t, q=q, G=G, sel=sel, phys=phys, **kw:
                     qs.quant_sparse_decode_attn(c, t, q, G, sel, phys, 30, **kw))
    want = [call() for call in calls]
    for i in rng.integers(0, len(calls), 60):
        out, lse = calls[i](workspace=ws)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
    assert qs.device_error() == 0


def test_one_long_request_over_all_multiprocessors():
    """A unit that every CTA has a part of, of 1 to 8 heads."""
    for G, d in ((1, 128), (8, 128), (2, 64), (8, 64)):
        _dense(quant_case(310 + G, [40000], h_kv=1, group=G, d=d, S=16))
    _sparse(quant_case(320, [60000], h_kv=1, group=2, d=64, S=16), 3500)


def test_without_lse_and_with_a_scale():
    import ctypes
    import query_aware_sparse_gb300 as qs
    case = quant_case(96, [333, 40], h_kv=2, group=2, d=64, S=16)
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    want, lse = qs.quant_dense_decode_attn(cache, t, q, 2, sm_scale=0.31)
    check_attention(np_of(want), np_of(lse), _reference(case, scale=float(np.float32(0.31))), 0.0, 0.0, 333)
    out = torch.empty_like(want)
    ws = torch.empty(qs.quant_decode_workspace_size(2, 2, 2, 64, 16), dtype=torch.uint8, device="cuda")
    st = qs.lib().quest_quant_dense_decode_attn(ctypes.byref(cache.quant), ctypes.byref(t.c), q.data_ptr(), 2, None,
                                                out.data_ptr(), None, ctypes.c_float(0.31), ws.data_ptr(), ws.numel(),
                                                torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(out, want)


@pytest.mark.parametrize("d,group", [(128, 2), (64, 8)])
def test_wait_runs_out_in_the_equal_runs(d, group):
    """Calls that are too long for a cluster per unit."""
    import query_aware_sparse_gb300 as qs
    case = quant_case(202, [20000, 300], h_kv=1, group=group, d=d, S=16)
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    _recovers(lambda: qs.quant_dense_decode_attn(cache, t, q, group),
              lambda o, l: check_attention(np_of(o), np_of(l), _reference(case), 0.0, 0.0, 20000))
    sel, phys = _lists(case, 1000, 7)
    dev = dev_i32(sel), dev_i32(phys)
    _recovers(lambda: qs.quant_sparse_decode_attn(cache, t, q, group, *dev, 1000),
              lambda o, l: check_attention(np_of(o), np_of(l), _sparse_reference(case, sel), 0.0, 0.0, 16000))


@pytest.mark.parametrize("d,group", [(128, 2), (64, 8)])
def test_wait_runs_out(d, group):
    import query_aware_sparse_gb300 as qs
    case = quant_case(201, [2000, 300, 40], h_kv=2, group=group, d=d, S=16)
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    _recovers(lambda: qs.quant_dense_decode_attn(cache, t, q, group),
              lambda o, l: check_attention(np_of(o), np_of(l), _reference(case), 0.0, 0.0, 2000))
    sel, phys = _lists(case, 60, 7)
    dev = dev_i32(sel), dev_i32(phys)
    _recovers(lambda: qs.quant_sparse_decode_attn(cache, t, q, group, *dev, 60),
              lambda o, l: check_attention(np_of(o), np_of(l), _sparse_reference(case, sel), 0.0, 0.0, 960))


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_decode_steps(fp8):
    """A prompt with normed, rotated keys into the E4M3 cache; a chunk of it
    attended through the read-back; then decode steps: append, score, select,
    sparse and dense attention, all against the fp64 forms on what is stored."""
    import query_aware_sparse_gb300 as qs
    import workloads as wl
    h, G, d, S, steps = 2, 4, 128, 16, 3
    lens = np.asarray([700, 45])
    table = wl.make_page_table(lens + steps, S, seed=5, permute=True, spare_pages=2)
    cache = qs.QuantCache.empty(table.n_phys, h, S, d, summary_fp8=fp8)
    cache.pool.fill_(0xff)
    g = torch.Generator(device="cuda").manual_seed(5)
    norm = qs.QKNorm(1 + 0.1 * torch.randn(d, generator=g, device="cuda"), 1 + 0.1 * torch.randn(d, generator=g, device="cuda"))
    inv = qs.rope_frequencies(d)
    scratch = qs.PagedCache.empty(table.nnz, h, S, d, F16)
    scratch.k_pool.fill_(float("nan"))
    scratch.v_pool.fill_(float("nan"))
    entries = np.arange(table.nnz, dtype=np.int32)

    def step(new, before):
        n = int(sum(new))
        qkv = torch.randn((n, (h * G + 2 * h), d), generator=g, device="cuda").half()
        seq = np.asarray(before) + np.asarray(new)
        t = gpu_table(table, seq_lens=seq.astype(np.int32))
        ind = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = qs.quant_append_kv(cache, t, qkv[:, :h * G], qkv[:, h * G:h * G + h], qkv[:, h * G + h:], dev_i32(ind), dev_i32(before),
                               G, inv_freq=inv, norm=norm)
        qs.quant_read_kv(cache, t, scratch)
        read = qs.PageTable(t.page_indptr, dev_i32(entries), t.seq_lens)
        assert qs.device_error() == 0
        pools = np_of(scratch.k_pool), np_of(scratch.v_pool)
        return q, t, read, seq, ind, pools

    q, t, read, seq, ind, pools = step(lens, [0, 0])
    out, lse = qs.prefill_attn(scratch, read, q, G, dev_i32(ind))
    ref = attention(np_of(q), *pools, table.page_indptr, entries, seq, ind, G)
    check_attention(np_of(out), np_of(lse), ref, 2.0 ** -11, 2.0 ** -11, 700)
    for i in range(steps):
        q, t, read, seq, ind, pools = step([1, 1], lens + i)
        ref = attention(np_of(q), *pools, table.page_indptr, entries, seq, ind, G)
        out, lse = qs.quant_dense_decode_attn(cache, t, q, G)
        check_attention(np_of(out), np_of(lse), ref, 0.0, 0.0, 703)
        scores = qs.score_pages(cache, t, q, G)
        # an upper bound of every stored key's product (up to the fp32 sums of both)
        k_all, qn, sc = pools[0].astype(np.float64), np_of(q).astype(np.float64), np_of(scores)
        for r in range(2):
            for p in range(-(-int(seq[r]) // S)):
                e = int(table.page_indptr[r]) + p
                cnt = min(S, int(seq[r]) - p * S)
                for kv in range(h):
                    dots = qn[r, kv * G:(kv + 1) * G] @ k_all[e, kv, :cnt].T
                    size = (np.abs(qn[r, kv * G:(kv + 1) * G]) @ np.abs(k_all[e, kv, :cnt]).T).max()
                    assert sc[kv, e] >= dots.max() - 2.0 ** -16 * size
        sel, phys, _ = qs.select_topk(t, h, S, scores, 12)
        out, lse = qs.quant_sparse_decode_attn(cache, t, q, G, sel, phys, 12)
        assert qs.device_error() == 0
        want, want_lse = qo.sparse_attention(np_of(q), *pools, table.page_indptr, entries, seq, np_of(sel), G)
        assert np.abs(np_of(out) - want).max() < 1e-4 and np.abs(np_of(lse) - want_lse).max() < 1e-4


def test_calls_that_need_fp16_pages_refuse_the_cache():
    import query_aware_sparse_gb300 as qs
    case = quant_case(97, [40], h_kv=1, group=1, d=64, S=16)
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    for call in (lambda: qs.dense_decode_attn(cache, t, q, 1), lambda: qs.prefill_attn(cache, t, q, 1, dev_i32([0, 1])),
                 lambda: qs.append_kv(cache, t, q, q, dev_i32([0, 1]), dev_i32([0])),
                 lambda: qs.sparse_decode_attn(cache, t, q, 1, None, None, 1)):
        with pytest.raises(TypeError):
            call()
    dst = qs.PagedCache.empty(8, 1, 32, 64, F16)
    with pytest.raises(ValueError):
        qs.quant_read_kv(cache, t, dst)
    with pytest.raises(ValueError):
        qs.quant_dense_decode_attn(cache, t, q.float(), 1)
    with pytest.raises(ValueError):
        qs.quant_sparse_decode_attn(cache, t, q, 1, dev_i32([[[0]]]), dev_i32([[0]]), 1)
    with pytest.raises(ValueError):
        qs.QuantCache(cache.pool[:, :, 16:], cache.summary, 16, 64)
    assert qs.device_error() == 0
