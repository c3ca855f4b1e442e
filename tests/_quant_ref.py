"""The E4M3 cache in plain numpy: quantising rows, the byte of a record that
holds a (token, dim), and cases whose pools hold records."""

from __future__ import annotations

import numpy as np
import torch

from tests._cases import np_of, random_case

TOP = 57344.0                           # 448 * 2^7


def quantise(x):
    """fp16 rows [..., d] -> (codes uint8, exponents e, row out of range)."""
    x = np.asarray(x, np.float16).astype(np.float64)
    over = (np.isnan(x) | (np.abs(x) > TOP)).any(-1)
    x = np.clip(np.where(np.isnan(x), 0.0, x), -TOP, TOP)
    top = np.abs(x).max(-1)
    e = np.full(top.shape, 7)
    for k in range(6, -15, -1):
        e = np.where(top <= 448.0 * 2.0 ** k, k, e)
    y = torch.from_numpy((x * 2.0 ** -e[..., None].astype(np.float64)).astype(np.float32))
    return y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), e, over


def stored(codes, e):
    """The fp16 numbers that codes and exponents stand for (checked to be such)."""
    c = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()
    x = c * 2.0 ** np.asarray(e, np.float64)[..., None]
    h = x.astype(np.float16)
    assert np.array_equal(h.astype(np.float64), x)
    return h


def k_at(S, d):
    """Byte of each (token, dim) of K in a record: [S, d]."""
    t, i = np.meshgrid(np.arange(S), np.arange(d), indexing="ij")
    return i // 64 * S * 64 + t * 64 + i % 64


def v_at(S, d):
    t, i = np.meshgrid(np.arange(S), np.arange(d), indexing="ij")
    lane = i % 32 // 4 * 4 + t % 8 // 2
    return S * d + ((t // 16 * (d // 32) + i // 32) * 32 + lane) * 16 + i % 4 * 4 + t % 16 // 8 * 2 + t % 2


def record(k, v):
    """Codes and exponents of K and V [..., S, d] -> records [..., 2 S (d + 1)]."""
    (kc, ke), (vc, ve) = k, v
    S, d = kc.shape[-2:]
    rec = np.zeros(kc.shape[:-2] + (2 * S * (d + 1),), np.uint8)
    rec[..., k_at(S, d)] = kc
    rec[..., v_at(S, d)] = vc
    rec[..., 2 * S * d:2 * S * d + S] = ke + 127
    rec[..., 2 * S * d + S:] = ve + 127
    return rec


def quant_case(seed, lens, garbage=0xFF, **shape):
    """random_case with `records` (bytes; `garbage` in slots without a token) and
    k_pool / v_pool replaced by the numbers that they hold."""
    case = random_case(seed, lens, **shape)
    return requantise(case, garbage)


def requantise(case, garbage=0xFF):
    S, d = case["S"], case["d"]
    parts = []
    for name in ("k_pool", "v_pool"):
        x = np_of(case[name])
        none = np.isnan(x).all(-1)
        c, e, _ = quantise(np.where(none[..., None], np.float16(0), x))
        parts.append((c, e))
        case[name] = torch.from_numpy(np.where(none[..., None], np.float16(np.nan), stored(c, e)))
    rec = record(*parts)
    fill(rec, none, garbage, S, d)
    case["records"], case["empty_slots"] = rec, none
    return case


def fill(rec, none, byte, S, d):
    """Bytes of the slots [n_phys, h, S] that hold no token."""
    p, h, s = np.nonzero(none)
    for at in (k_at(S, d), v_at(S, d)):
        rec[p[:, None], h[:, None], at[s]] = byte
    rec[p, h, 2 * S * d + s] = byte
    rec[p, h, 2 * S * d + S + s] = byte


def gpu_quant(case, summary=None):
    import query_aware_sparse_gb300 as qs
    rec = torch.from_numpy(case["records"]).cuda()
    sm = torch.zeros((rec.shape[0], rec.shape[1], 2, case["d"]), dtype=torch.float16) if summary is None else summary
    return qs.QuantCache(rec, sm.cuda().contiguous(), case["S"], case["d"])
