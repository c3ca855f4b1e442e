"""Prompt attention's paths (one row tile per CTA and two, keys whole and cut into
parts) with every mask, bias and cap: rows here and there in 64 bits."""

import math

import numpy as np
import pytest
import torch

from tests._cases import F16, dev_i32, gpu_cache, gpu_table
from tests.test_gpu_dense import HALF16, _rows_case

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
# lens, rows, KV heads, group, keys cut
SHAPES = {"one": ([700, 33, 900], [700, 3, 900], 2, 4, False),
          "one_cut": ([6000, 0, 2500], [33, 0, 5], 2, 1, True),
          "two": ([8300, 8700], [8300, 8650], 1, 8, False),
          "two_cut": ([9000, 17003], [520, 300], 1, 2, True)}
KINDS = ["", "cap", "alibi", "doc", "prefix", "window", "bad", "cap alibi", "cap doc prefix", "alibi window bad",
         "cap alibi doc prefix window bad"]


def _row(case, mods, ids, r, i, softcap):
    """Row i of request r in 64 bits, all heads: (out, lse, error bounds of both), or
    None if it sees nothing."""
    L, rows, G, d = int(case["table"].seq_lens[r]), case["rows"][r], case["group"], case["d"]
    S, n = case["S"], case["gpu"]
    p = L - rows + i
    at = int(case["q_indptr"][r]) + i
    lo = max(0, p - mods["window"] + 1) if mods["window"] else 0
    lo = max(lo, int(mods["doc"][at])) if mods["doc"] is not None else lo
    hi = min(L, max(p + 1, int(mods["prefix"][r]))) if mods["prefix"] is not None else p + 1
    j = torch.arange(lo, hi, device="cuda")
    page = ids[j // S]
    j, page = j[page >= 0], page[page >= 0]
    if len(j) == 0:
        return None
    k, v = (n[x][page, :, j % S].double() for x in ("k", "v"))              # [keys, h_kv, d]
    q = n["q"][at].double().view(-1, G, d)
    x = torch.einsum("hgd,jhd->hgj", q, k) / math.sqrt(d)
    # fp32 dot of d terms and the scale; tanh to 16 units of 2^-24 of the logit or, for
    # caps up to 64, 2^-21 of the cap; the bias; base 2 and the maximum
    err = (d + 4) * EPS * torch.einsum("hgd,jhd->hgj", q.abs(), k.abs()) / math.sqrt(d)
    if softcap:
        x = softcap * torch.tanh(x / softcap)
        err = err + 16 * EPS * x.abs() + 2.0 ** -21 * softcap
    if mods["slopes"] is not None:
        far = mods["slopes"].double().view(-1, G, 1) * (p - j).abs()
        x = x - far
        err = err + 4 * EPS * (far + x.abs())
    m = x.amax(-1, keepdim=True)
    dx = torch.where(x > m - 40, err + 6 * EPS * (x.abs() + m.abs() + 1), 0.0).amax(-1) + 2.0 ** -20
    w = torch.exp(x - m)
    total = w.sum(-1)
    o, mean = (torch.einsum("hgj,jhd->hgd", w, y) / total[..., None] for y in (v, v.abs()))
    lse = m[..., 0] + total.log()
    # a row's sums: 16 keys a step lose 5 units of 2^-24 at most, for at most 8192 keys
    # (then fp32), a fp32 sum per 64 keys; weights below fp16's range 2^-24 2^-6 each
    sums = (5 * min(len(j), 8192) / 16 + len(j) / 64 + 64) * EPS
    tol_o = (2 * dx[..., None] + HALF16 + sums) * mean + HALF16 * o.abs() + len(j) * EPS * 2.0 ** -6 * v.abs().max() + 2.0 ** -25
    tol_l = dx + (len(j) / 64 + 64) * EPS + 2.0 ** -22 * lse.abs()
    return o.reshape(-1, d), lse.reshape(-1), tol_o.reshape(-1, d), tol_l.reshape(-1)


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("d,S", [(64, 32), (128, 16)])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_prefill_paths(shape, d, S, kinds):
    import query_aware_sparse_gb300 as qs
    lens, rows, h, G, cut = SHAPES[shape]
    kinds = kinds.split()
    case = _rows_case(500 + d, lens, rows, h_kv=h, group=G, d=d, S=S)
    t, hq, n = case["table"], h * G, sum(rows)
    rng = np.random.default_rng(d + len(kinds))
    mods = dict(window=5000 if "window" in kinds else 0, doc=None, prefix=None, slopes=None)
    if "doc" in kinds:
        at = np.concatenate([np.arange(L - r, L) for L, r in zip(lens, rows)])
        mods["doc"] = (at // 3001 * 3001).astype(np.int32)
    if "prefix" in kinds:
        mods["prefix"] = rng.integers(0, 5000, len(lens)).astype(np.int32)
    if "alibi" in kinds:
        mods["slopes"] = torch.as_tensor(2.0 ** -rng.uniform(2, 12, hq), dtype=torch.float32, device="cuda")
    if "bad" in kinds:
        for r, L in enumerate(lens):
            for p in rng.integers(0, max(1, L // S), 3 if L > 100 else 0):
                t.page_indices[t.page_indptr[r] + p] = t.n_phys + int(p) if p & 1 else -1 - int(p)
    cache, table = gpu_cache(case["k_pool"], case["v_pool"], case["summary"]), gpu_table(t)
    case["gpu"] = dict(k=cache.k_pool, v=cache.v_pool, q=case["q"].cuda())
    need = qs.prefill_workspace_size(len(lens), n, table.nnz, h, G, d, S, F16)
    assert (need > 2 * n * hq * d * 4) == cut
    ids = [torch.as_tensor(t.page_indices[t.page_indptr[r]:t.page_indptr[r + 1]].astype(np.int64), device="cuda")
           for r in range(len(lens))]
    ids = [torch.where((x >= 0) & (x < t.n_phys), x, -1) for x in ids]
    for softcap in (3.0, 50.0) if "cap" in kinds else (0.0,):
        m = qs.ScoreMods(softcap=softcap, window=mods["window"], alibi_slopes=mods["slopes"],
                         doc_starts=None if mods["doc"] is None else dev_i32(mods["doc"]),
                         prefix_lens=None if mods["prefix"] is None else dev_i32(mods["prefix"]))
        out, lse = qs.prefill_attn(cache, table, case["gpu"]["q"], G, dev_i32(case["q_indptr"]), mods=m)
        assert qs.device_error() == ("bad" in kinds)
        assert torch.isfinite(out).all()
        for r, k in enumerate(rows):
            for i in sorted({x for x in (0, 1, 15, 16, 31, 32, 127, 128, 255, 256, 3000, 3001, k // 2, k - 2, k - 1) if 0 <= x < k}):
                at, want = int(case["q_indptr"][r]) + i, _row(case, mods, ids[r], r, i, softcap)
                if want is None:
                    assert (out[at] == 0).all() and torch.isneginf(lse[at]).all()
                    continue
                o, z, tol_o, tol_l = want
                e = (out[at].double() - o).abs()
                assert (e <= tol_o).all(), (softcap, r, i, float((e / tol_o).max()))
                e = (lse[at].double() - z).abs()
                assert (e <= tol_l).all(), (softcap, r, i, float((e / tol_l).max()))
