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
