"""Sums over many keys whose exact mean lies between two fp16 numbers, for some dims
close to the middle, where a small error of the sum shows in the rounded output."""

import math

import numpy as np
import pytest
import torch

from tests._cases import F16, dev_i32

pytestmark = pytest.mark.gpu

# batch (all requests on the same pages), keys, rows per request, KV heads, group, page,
# keys cut into parts: two row tiles and one, whole and cut
SHAPES = [(1, 65536, 16384, 4, 1, 16, False), (1, 40007, 20000, 4, 4, 32, False), (1, 131072, 512, 8, 4, 16, True),
          (200, 65536, 4, 8, 4, 16, False), (400, 30001, 1, 8, 8, 32, False), (1, 131072, 3, 4, 8, 16, True),
          (1, 9000, 9000, 8, 1, 16, False)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_prefill_sums(shape, d):
    """Every row sees every key. Every 61st key has the largest logit, the others one
    that makes their weights 2^6 * 1585 / 2048, a number of eleven bits; the values have
    eleven bits as well."""
    import query_aware_sparse_gb300 as qs
    batch, L, rows, h, group, S, cut = shape
    pages = -(-L // S)
    g = torch.Generator(device="cuda").manual_seed(L + d)
    j = torch.arange(pages * S, device="cuda", dtype=torch.float64)
    top = j % 61 == 0
    share = torch.linspace(0.3, 0.7, d, dtype=torch.float64, device="cuda")
    upper = (j * 0.6180339887498949 % 1.0)[:, None] < share[None]             # [keys, d], even along the keys
    base = 1.0 + torch.randint(0, 1022, (d,), generator=g, device="cuda").double() * 2.0 ** -10
    v = (base + upper.double() * 2.0 ** -10).half()
    k = torch.zeros((pages * S, d), dtype=F16, device="cuda")
    k[top, 0] = 1.0
    ids = torch.randperm(pages, generator=g, device="cuda")
    kp, vp = (torch.empty((pages, h, S, d), dtype=F16, device="cuda") for _ in range(2))
    kp[ids], vp[ids] = k.view(pages, 1, S, d).expand(-1, h, -1, -1), v.view(pages, 1, S, d).expand(-1, h, -1, -1)
    cache = qs.PagedCache(kp, vp, torch.zeros((pages, h, 2, d), dtype=F16, device="cuda"))
    table = qs.PageTable(dev_i32(np.arange(batch + 1) * pages), ids.to(torch.int32).repeat(batch), dev_i32([L] * batch))
    q = torch.zeros((batch * rows, h * group, d), dtype=F16, device="cuda")
    q[..., 0] = 1.0
    size = qs.prefill_workspace_size(batch, batch * rows, batch * pages, h, group, d, S, F16)
    assert (size > 2 * batch * rows * h * group * d * 4) == cut
    out, lse = qs.prefill_attn(cache, table, q, group, dev_i32(np.arange(batch + 1) * rows),
                               sm_scale=math.log(2048 / 1585), mods=qs.ScoreMods(prefix_lens=dev_i32([L] * batch)))
    assert qs.device_error() == 0
    w = 1.0 + (2048 / 1585 - 1.0) * top[:L].double()
    mean = (w @ (base + upper[:L].double() * 2.0 ** -10)) / w.sum()
    # The output's rounding, half a step of 2^-10, and the sums'. An accumulator takes
    # 16 keys with each term cut to a quarter of its last place and the result to one,
    # 16 / 8 + 1 / 2 places lost on average of uniform low bits; a place is 2^-23 of it
    # at most, half of that over a chain that grows evenly: 512 steps of 8192 keys lose
    # 640 2^-23, a little less than 2^-13. The weights' sum takes a rounding of 2^-24 per
    # 64 keys, the parts' join 64, the logit and its exponential 2^-20.
    total = (L / 64 + 64) * 2.0 ** -24 + 2.0 ** -20
    tol = 2.0 ** -11 + mean * (2.0 ** -13 + total)
    err = (out.view(-1, d).double() - mean).abs()
    assert (err <= tol).all(), float(((err - 2.0 ** -11) / mean).max())
    assert ((lse.double() - w.sum().log()).abs() <= total + 2.0 ** -22 * 12).all()


def _shared(batch, L, rows, h, group, d, S, seed):
    """Requests of L tokens on the same pages, `rows` query rows each."""
    from types import SimpleNamespace

    import query_aware_sparse_gb300 as qs
    pages = -(-L // S)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").half()
    kp, vp, ids = rand(pages, h, S, d), rand(pages, h, S, d), torch.randperm(pages, generator=g, device="cuda")
    cache = qs.PagedCache(kp, vp, torch.zeros((pages, h, 2, d), dtype=F16, device="cuda"))
    table = qs.PageTable(dev_i32(np.arange(batch + 1) * pages), ids.to(torch.int32).repeat(batch), dev_i32([L] * batch))
    q = rand(batch * rows, h * group, d)
    case = dict(table=SimpleNamespace(seq_lens=np.full(batch, L)), rows=[rows] * batch, group=group, d=d, S=S,
                q_indptr=np.arange(batch + 1) * rows, gpu=dict(k=kp, v=vp, q=q))
    return case, cache, table, ids


# requests, keys, rows each, KV heads, group, page: one row tile and two, chains of 8192 keys and what is left
LONG = [(120, 17000, 3, 4, 4, 16), (1, 20000, 9000, 4, 2, 32), (2, 30001, 15000, 2, 4, 16)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", LONG)
def test_long_rows_under_masks(shape, d):
    from tests.test_gpu_dense_paths import _row
    import query_aware_sparse_gb300 as qs
    batch, L, rows, h, group, S = shape
    case, cache, table, ids = _shared(*shape[:5], d, S, L + d)
    at = np.tile(np.arange(L - rows, L), batch)
    rng = np.random.default_rng(L)
    slopes = torch.as_tensor(2.0 ** -rng.uniform(8, 14, h * group), dtype=torch.float32, device="cuda")
    for softcap, window, doc, prefix, bias in ((0.0, 0, None, None, None), (50.0, 16000, None, None, slopes),
                                               (3.0, 0, at // 7000 * 4000, np.full(batch, 12345), None)):
        mods = dict(window=window, doc=doc, prefix=prefix, slopes=bias)
        m = qs.ScoreMods(softcap=softcap, window=window, alibi_slopes=bias,
                         doc_starts=None if doc is None else dev_i32(doc),
                         prefix_lens=None if prefix is None else dev_i32(prefix))
        out, lse = qs.prefill_attn(cache, table, case["gpu"]["q"], group, dev_i32(case["q_indptr"]), mods=m)
        for r, i in ((0, 0), (batch - 1, rows - 1), (batch // 2, rows // 2), (0, min(rows - 1, 255)), (batch - 1, rows // 3)):
            o, z, tol_o, tol_l = _row(case, mods, ids, r, i, softcap)
            e = (out[r * rows + i].double() - o).abs()
            assert (e <= tol_o).all(), (softcap, r, i, float((e / tol_o).max()))
            e = (lse[r * rows + i].double() - z).abs()
            assert (e <= tol_l).all(), (softcap, r, i, float((e / tol_l).max()))
    assert qs.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", LONG)
def test_long_rows_repeat_bit_for_bit(shape, d):
    """Whatever stands in the workspace, on another stream, captured and replayed."""
    import query_aware_sparse_gb300 as qs
    batch, L, rows, h, group, S = shape
    case, cache, table, _ = _shared(*shape[:5], d, S, L + d)
    q, ind = case["gpu"]["q"], dev_i32(case["q_indptr"])
    size = qs.prefill_workspace_size(batch, batch * rows, table.nnz, h, group, d, S, F16)
    space = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = qs.prefill_attn(cache, table, q, group, ind, workspace=space)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    same = lambda: torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for fill in (0xff, 0x7b, 0x3c):                    # NaN, large numbers, ordinary ones
        space.fill_(fill)
        qs.prefill_attn(cache, table, q, group, ind, out=out, lse=lse, workspace=space)
        assert same(), fill
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qs.prefill_attn(cache, table, q, group, ind, out=out, lse=lse, workspace=space, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qs.prefill_attn(cache, table, q, group, ind, out=out, lse=lse, workspace=space)
    for _ in range(3):
        out.zero_()
        space.fill_(0xff)
        graph.replay()
        assert same()
    assert qs.device_error() == 0
