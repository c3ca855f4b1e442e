"""Capped scores over the whole range of caps, on every path of the attention
calls: each row sees one key, itself, so its lse is that key's capped logit."""

import numpy as np
import pytest
import torch

from tests._cases import F16, F32, dev_i32, gpu_cache, gpu_table, np_of
from tests.test_gpu_dense import _rows_case

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
CAPS = [1e-3, 3.0, 50.0, 1e4, 1e6, 1e10, 1e30, 3e38]

# lens, rows, KV heads, group, whether each row block's keys are cut into parts:
# one row tile per CTA, and two (from a mean of 4096 keys on), each whole and cut
SHAPES = {"one": ([700, 90], [700, 90], 2, 2, False),
          "one_cut": ([6000], [33], 1, 4, True),
          "two": ([8300], [8300], 1, 8, False),
          "two_cut": ([9000], [520], 1, 2, True)}


def _case(shape, d, dtype, seed):
    """Queries of 2^-5 to 32 times the usual size: runs of 160 tokens whose logits
    are below one, and runs where they are of every size, side by side."""
    lens, rows, h, group, _ = SHAPES[shape]
    case = _rows_case(seed, lens, rows, h_kv=h, group=group, d=d, S=16, dtype=dtype)
    g = torch.Generator().manual_seed(seed)
    n, hq = sum(rows), h * group
    low = (torch.arange(n) // 160 % 2 == 0)[:, None]
    size = torch.where(low, -5 + 3 * torch.rand((n, hq), generator=g), -5 + 10 * torch.rand((n, hq), generator=g))
    case["q"] = (case["q"].float() * 2.0 ** size[..., None]).to(dtype)
    at = np.concatenate([np.arange(L - r, L) for L, r in zip(lens, rows)])
    own = np.concatenate([case["tok_indptr"][i] + np.arange(L - r, L) for i, (L, r) in enumerate(zip(lens, rows))])
    case["at"], case["own"] = at.astype(np.int32), own
    return case


def _expected(case, rows, cap):
    """lse in 64 bits and its error bound: the dot product of d terms in fp32, the
    scale, tanh to 16 units of 2^-24 of the CAPPED LOGIT, whatever the cap, then the
    logarithm and the sums that follow. Caps up to 64 may go by 1 - 2 / (1 + e^y):
    near y = 0 an exponential to 2^-22, a sum of 2 to 2^-24 and a reciprocal to
    2^-23 of themselves make 2 (2^-23 + 2^-24 + 2^-23) / 2 < 2^-21 of the cap."""
    d = case["d"]
    q = np_of(case["q"]).astype(np.float64)[rows]
    k = np_of(case["k_tok"]).astype(np.float64)[case["own"][rows]].repeat(case["group"], axis=1)
    x = (q * k).sum(-1) / np.sqrt(d)
    err = (d + 4) * EPS * (np.abs(q) * np.abs(k)).sum(-1) / np.sqrt(d)
    y = cap * np.tanh(x / cap)
    if cap <= 64:
        err = err + 2.0 ** -21 * cap
    tol = err + 16 * EPS * np.abs(y) + 6 * EPS * (2 * np.abs(y) + 1) + 2.0 ** -20 + 2.0 ** -22 * np.abs(y)
    return y, tol


def _compare(case, out, lse, rows, cap, half):
    want, tol = _expected(case, rows, cap)
    err = np.abs(np_of(lse).astype(np.float64) - want)
    assert (err <= tol).all(), (cap, float((err / tol).max()), float(err.max()))
    # the weight (as o and as l) and the output, each rounded once
    v = np_of(case["v_tok"]).astype(np.float64)[case["own"][rows]].repeat(case["group"], axis=1)
    got = np_of(out).astype(np.float64)
    assert (np.abs(got - v) <= (2 * half + 2.0 ** -20) * np.abs(v) + 2.0 ** -24).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_prefill_caps(shape, d):
    import query_aware_sparse_gb300 as qs
    lens, rows, h, group, cut = SHAPES[shape]
    case = _case(shape, d, F16, 300 + d)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    need = qs.prefill_workspace_size(len(lens), sum(rows), table.nnz, h, group, d, 16, F16)
    assert (need > 2 * sum(rows) * h * group * d * 4) == cut     # more than one part of all rows
    q, ind, docs = case["q"].cuda(), dev_i32(case["q_indptr"]), dev_i32(case["at"])
    every = np.arange(sum(rows))
    for cap in CAPS:
        out, lse = qs.prefill_attn(cache, table, q, group, ind, mods=qs.ScoreMods(softcap=cap, doc_starts=docs))
        _compare(case, out, lse, every, cap, 2.0 ** -11)
    assert qs.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_caps_f32(d):
    import query_aware_sparse_gb300 as qs
    case = _case("one", d, F32, 310 + d)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    q, ind, docs = case["q"].cuda(), dev_i32(case["q_indptr"]), dev_i32(case["at"])
    for cap in CAPS:
        out, lse = qs.prefill_attn(cache, table, q, 2, ind, mods=qs.ScoreMods(softcap=cap, doc_starts=docs))
        _compare(case, out, lse, np.arange(790), cap, 2.0 ** -22)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_caps(d, dtype):
    """The same logits from the call of one new token."""
    import query_aware_sparse_gb300 as qs
    case = _case("one", d, dtype, 320 + d)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    for cap in CAPS:
        for last in ([699, 789], [13, 710], [200, 750]):
            lens = np.asarray([last[0] + 1, last[1] - 699], np.int32)
            out, lse = qs.dense_decode_attn(cache, gpu_table(case["table"], seq_lens=lens), case["q"][last].cuda(), 2,
                                            mods=qs.ScoreMods(softcap=cap, window=1))
            _compare(case, out, lse, np.asarray(last), cap, 2.0 ** -22)
    assert qs.device_error() == 0


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,rows,group,cut", [(704, 704, 2, False), (6016, 33, 4, True), (8320, 8320, 8, False),
                                              (9088, 520, 2, True)])
def test_prefill_caps_of_whole_blocks(L, rows, group, cut, d, alibi):
    """Every row sees every key, all of them equal: lse is the capped logit and the
    logarithm of the keys' number (of the sum of their biases). Runs of 160 tokens
    of small, of middling and of mixed logits."""
    import query_aware_sparse_gb300 as qs
    case = _rows_case(330 + d, [L], [rows], h_kv=1, group=group, d=d, S=16, spare=0)
    key = case["k_tok"][0, 0]
    case["k_pool"][:] = key
    g = torch.Generator().manual_seed(d)
    run = torch.arange(rows) // 160 % 3
    size = torch.rand((rows, group), generator=g)
    size = torch.where((run == 0)[:, None], -5 + 4 * size, torch.where((run == 1)[:, None], 3 * size, -5 + 11 * size))
    case["q"] = (torch.sign(case["q"].float()) * torch.sign(key.float()) * torch.sign(torch.rand((rows, group, 1), generator=g) - 0.3)
                 * torch.rand(case["q"].shape, generator=g) * 2.0 ** (size[..., None] - 3)).half()
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(case["table"])
    assert (qs.prefill_workspace_size(1, rows, table.nnz, 1, group, d, 16, F16) > 2 * rows * group * d * 4) == cut
    slopes = (2.0 ** -np.arange(1, group + 1)).astype(np.float32)
    far = np.abs(np.arange(L - rows, L)[:, None] - np.arange(L)[None])
    bias = np.stack([np.log(np.exp(-float(s) * far).sum(1)) for s in slopes], 1) if alibi else np.log(L)
    q, k = np_of(case["q"]).astype(np.float64), np_of(key).astype(np.float64)
    x, size = q @ k / np.sqrt(d), np.abs(q) @ np.abs(k) / np.sqrt(d)
    for cap in CAPS:
        mods = qs.ScoreMods(softcap=cap, prefix_lens=dev_i32([L]),
                            alibi_slopes=torch.as_tensor(slopes, device="cuda") if alibi else None)
        out, lse = qs.prefill_attn(cache, table, case["q"].cuda(), group, dev_i32([0, rows]), mods=mods)
        y = cap * np.tanh(x / cap)
        tol = (d + 4) * EPS * size + (16 * np.abs(y) + 6 * (2 * np.abs(y) + 41)) * EPS + 2.0 ** -20 + 2.0 ** -22 * np.abs(y + bias)
        if cap <= 64:
            tol = tol + 2.0 ** -21 * cap
        tol = tol + (L / 16 + 64) * EPS                # the sum of L weights
        err = np.abs(np_of(lse).astype(np.float64) - (y + bias))
        assert (err <= tol).all(), (cap, float((err / tol).max()), float(err.max()))
    assert qs.device_error() == 0
