"""What a weight keeps on its way through the tensor core: two fp16 numbers,
2^-22 of itself from 2^-9 of the largest on, 2^-31 of the largest below."""

import numpy as np
import pytest
import torch

from tests._cases import F16, dev_i32, gpu_cache, gpu_table, np_of, random_case
from tests._quant_ref import gpu_quant, requantise
from tests.test_gpu_quant_decode import _lists, _reference, _sparse_reference

pytestmark = pytest.mark.gpu


def _check(out, ref, mass, n_keys):
    """mass: the sum of |V| over the row's keys, per dim. A weight is off by at most
    2^-25 where the largest is 2^6 at least (and by 2^-33 more where it was split
    twice, the first time under a maximum 2^8 lower): 2^-31 of the largest. Logits
    are single products of small numbers here, so what else a weight is off by is
    relative: in base 2 two roundings of numbers below 64 (2^-18 ln 2 together) and
    ex2 (2^-21); sums as in check_attention."""
    rel = 2.0 ** -18 + 2.0 ** -21 + 2.0 ** -22 + (n_keys / 16 + 64) * 2.0 ** -24
    tol = 2 * rel * ref["aw"] + 1.01 * 2.0 ** -31 * mass + 2.0 ** -25
    err = np.abs(np_of(out).astype(np.float64) - ref["out"])
    assert np.all(err <= tol), float((err / tol).max())


def _mass(case, sel=None):
    """[batch, heads, d]: sums of |V| over a request's tokens, or a list's."""
    t, h, G, S = case["table"], case["h_kv"], case["group"], case["S"]
    v = np.abs(np_of(case["v_pool"]).astype(np.float64))
    out = np.zeros((t.batch, h * G, case["d"]))
    for r in range(t.batch):
        L = int(t.seq_lens[r])
        for g in range(h):
            pages = np.arange(-(-L // S)) if sel is None else sel[r, g][sel[r, g] >= 0]
            for p in pages:
                rows = v[t.page_indices[t.page_indptr[r] + p], g, :min(S, L - int(p) * S)]
                out[r, g * G:(g + 1) * G] += rows.sum(0)
    return out


def _uneven(seed, group, d, S, quant):
    """A token of weight 1 and many of e^-7, with small values, and tokens of
    weights from e^-10 down to e^-20 whose values are 2^17 times larger. A query
    head is 1 in a dim of its own, where the keys hold its logits."""
    case = random_case(seed, [300, 77], h_kv=2, group=group, d=d, S=S)
    rng = np.random.default_rng(seed)
    t = case["table"]
    case["q"].zero_()
    for h in range(2 * group):
        case["q"][:, h, h % group] = 1.0
    for r in range(2):
        L = int(t.seq_lens[r])
        pp, at = t.page_indices[t.page_indptr[r] + np.arange(L) // S], np.arange(L) % S
        x = np.zeros((2, d, L))
        big = np.zeros((2, L), bool)
        for g in range(2):
            big[g, rng.permutation(L)[:40]] = True
            for c in range(group):
                x[g, c] = np.where(big[g], -rng.choice([10, 11, 12, 13, 14, 15, 16, 18, 20], L), -7.0)
                x[g, c, rng.choice(np.nonzero(~big[g])[0])] = 0.0
        case["k_pool"][pp, :, at] = torch.from_numpy(x.transpose(2, 0, 1)).half()
        v = rng.normal(size=(L, 2, d)).clip(-3.4, 3.4) * np.where(big.T, 2.0 ** 13, 2.0 ** -4)[:, :, None]
        case["v_pool"][pp, :, at] = torch.from_numpy(v).half()
    if quant:
        requantise(case)
    return case


@pytest.mark.parametrize("d,S,group", [(128, 16, 2), (64, 32, 4), (64, 16, 8), (128, 32, 8), (128, 32, 1)])
def test_e4m3_cache(d, S, group):
    import query_aware_sparse_gb300 as qs
    case = _uneven(500 + group, group, d, S, True)
    cache, t, q = gpu_quant(case), gpu_table(case["table"]), case["q"].cuda()
    out, _ = qs.quant_dense_decode_attn(cache, t, q, group, sm_scale=1.0)
    _check(out, _reference(case, scale=1.0), _mass(case), 300)
    sel, phys = _lists(case, 9, 0)
    out, _ = qs.quant_sparse_decode_attn(cache, t, q, group, dev_i32(sel), dev_i32(phys), 9, sm_scale=1.0)
    _check(out, _sparse_reference(case, sel, scale=1.0), _mass(case, sel), 9 * S)
    assert qs.device_error() == 0


@pytest.mark.parametrize("d,S,group", [(128, 16, 2), (64, 32, 4)])
def test_fp16_cache(d, S, group):
    import query_aware_sparse_gb300 as qs
    case = _uneven(510 + group, group, d, S, False)
    sm = torch.zeros((case["k_pool"].shape[0], 2, 2, d), dtype=F16)
    out, _ = qs.dense_decode_attn(gpu_cache(case["k_pool"], case["v_pool"], sm), gpu_table(case["table"]),
                                  case["q"].cuda(), group, sm_scale=1.0)
    _check(out, _reference(case, scale=1.0), _mass(case), 300)
    assert qs.device_error() == 0
