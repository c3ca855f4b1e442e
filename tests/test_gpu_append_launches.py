"""The normed and the E4M3 append in every launch that csrc/norm_append.cu and
norm_append.cuh choose between: CTAs of eight warps and of four, steps of 16
tokens and of a few, KV heads in more parts for much work. Sizes come from the
device's SM count."""

import numpy as np
import pytest
import torch

from tests import test_gpu_norm_append as plain
from tests import test_gpu_quant_append as quant
from tests._cases import F16, F32

pytestmark = pytest.mark.gpu

SHAPES = [(128, 16), (64, 32), (64, 16), (128, 32)]


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def launch(n_new, batch, h, S, d, group=0, size=2):
    """(warps of a CTA, steps of few tokens, parts of the KV heads), as chosen
    there; group 0: no queries."""
    sms = _sms()
    much = h * (group + 2) * n_new * d * size // 4096 > 6 * 16 * sms
    pages = min(n_new, -(-n_new // S) + 2 * batch)
    heads = h
    while heads > 1 and pages * -(-h // heads) < (5 if much else 1) * sms:
        heads = (heads + 1) // 2
    parts = -(-h // heads)
    return 4 if pages * parts > 4 * sms else 8, n_new <= 4 * batch, parts, much


def _long(S):
    """Two requests whose pages are more than four per SM."""
    return [(4 * _sms() + 9) * S, 19], [5, 40]


def _many(seed):
    """A token each for most, none for some, a page of them for one: more than
    four pages per SM, few tokens per request."""
    rng = np.random.default_rng(seed)
    lens = np.ones(4 * _sms() + 50, int)
    lens[rng.permutation(len(lens))[:30]] = 0
    lens[rng.permutation(len(lens))[:40]] = 3
    lens[7] = 50
    return lens.tolist(), rng.integers(0, 50, len(lens)).tolist()


@pytest.mark.parametrize("d,S", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("treated", [False, True])
def test_e4m3_long(d, S, fp8, treated):
    lens, before = _long(S)
    assert launch(sum(lens), 2, 1, S, d, 2 * treated) == (4, False, 1, False)
    quant._check(21, lens, before, h=1, d=d, S=S, fp8=fp8, rope=treated, norm=treated, interleaved=treated and fp8)


@pytest.mark.parametrize("d,S", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("treated", [False, True])
def test_e4m3_many_short(d, S, fp8, treated):
    lens, before = _many(S)
    assert launch(sum(lens), len(lens), 2, S, d, 2 * treated) == (4, True, 1, False)
    quant._check(22, lens, before, d=d, S=S, fp8=fp8, rope=treated, norm=treated, interleaved=treated and fp8)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,fp8", [(F16, False), (F16, True), (F32, False)])
@pytest.mark.parametrize("d,S", [(128, 16), (64, 32)])
def test_plain_long(d, S, dtype, fp8, interleaved):
    lens, before = _long(S)
    assert launch(sum(lens), 2, 1, S, d, 1, 2 if dtype == F16 else 4) == (4, False, 1, False)
    plain._check(23, lens, before, h=1, group=1, d=d, S=S, dtype=dtype, fp8=fp8, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,fp8", [(F16, False), (F16, True), (F32, False)])
@pytest.mark.parametrize("d,S", [(128, 16), (64, 32)])
def test_plain_many_short(d, S, dtype, fp8, interleaved):
    lens, before = _many(S + 1)
    assert launch(sum(lens), len(lens), 2, S, d, 2, 2 if dtype == F16 else 4) == (4, True, 1, False)
    plain._check(24, lens, before, d=d, S=S, dtype=dtype, fp8=fp8, interleaved=interleaved, per_head=interleaved)


def test_heads_in_more_parts_for_much_work():
    """Enough pages for a CTA per SM with all KV heads in one; over the limit
    of steps the heads are spread further."""
    rows = 6 * 16 * _sms() * 4096 // 256           # of 256 bytes, just at the limit
    for h, group in ((40, 1), (9, 8)):
        n = rows // (h * (group + 2)) + 20
        assert launch(n, 1, h, 16, 128, group) == (4, False, launch(n, 1, h, 16, 128, group)[2], True)
        assert launch(n, 1, h, 16, 128, group)[2] > launch(n - 40, 1, h, 16, 128, group)[2]
        quant._check(25, [n], [3], h=h, group=group, rope=True, norm=True)
        plain._check(26, [n], [3], h=h, group=group, fp8=True)
    n = rows // (40 * 3) + 20
    assert launch(n, 1, 40, 32, 64, 1, 4)[3] and launch(n, 1, 40, 32, 64, 1, 4)[2] > 1
    plain._check(27, [n], [3], h=40, group=1, d=64, S=32, dtype=F32, interleaved=True)


@pytest.mark.parametrize("e4m3", [False, True])
def test_repeats_bit_for_bit(e4m3):
    """A long prompt over and over, into pages that hold something else before."""
    import query_aware_sparse_gb300 as qs
    h, group, d, S = 2, 4, 128, 16
    n = (4 * _sms() + 9) * S + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((n, h * (group + 2), d), generator=g, device="cuda").half()
    q, k, v = x[:, :h * group], x[:, h * group:h * (group + 1)], x[:, h * (group + 1):]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = -(-n // S)
    table = qs.PageTable(i32(0, pages), torch.randperm(pages, generator=g, device="cuda").to(torch.int32), i32(n))
    weight = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    norm, inv, out = qs.QKNorm(weight, weight), qs.rope_frequencies(d), torch.empty((n, h * group, d), dtype=F16, device="cuda")
    if e4m3:
        cache = qs.QuantCache.empty(pages, h, S, d, summary_fp8=True)
        state = (cache.pool, cache.summary, out)
    else:
        cache = qs.PagedCache.empty(pages, h, S, d, F16, summary_fp8=True)
        state = (cache.k_pool, cache.v_pool, cache.summary, out)
    want = None
    for byte in (0, 0x41, 0xff, 0x80, 0x7e, 0x13):
        for t in state:
            t.view(torch.uint8).fill_(byte)
        if e4m3:
            qs.quant_append_kv(cache, table, q, k, v, i32(0, n), i32(0), group, inv_freq=inv, norm=norm, q_out=out)
        else:
            qs.norm_rope_append_kv(cache, table, q, k, v, i32(0, n), i32(0), norm, group, inv_freq=inv, q_out=out)
        # slots behind the last token hold what they held
        tail = table.page_indices[-1].long()
        got = [t.view(torch.uint8).clone() for t in state]
        for t in got[:-1]:
            if t.dim() > 1 and t.shape[0] == pages and not (t.shape[2] == 2 and t.dim() == 4):
                t[tail] = 0
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert qs.device_error() == 0
