"""Plain fp64 forms of the dense-layer operators (rotating append, dense decode
and prompt attention) and the error bounds their tests use."""

from __future__ import annotations

import math

import numpy as np


def rotate(x, pos, inv_freq, interleaved):
    """Rotary embedding in fp64: x [n, heads, d], pos [n]. Returns (y, size):
    size bounds |x_a| + |x_b| of every output's pair (0 where nothing turns)."""
    y = x.astype(np.float64).copy()
    half = len(inv_freq)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    # long double where the platform has one changes nothing at these sizes:
    # the angle is below 2^32 radians, its fp64 rounding below 2^-20 of one
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    xa, xb = x[..., a].astype(np.float64), x[..., b].astype(np.float64)
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    size = np.zeros_like(y)
    size[..., a] = size[..., b] = np.abs(xa) + np.abs(xb)
    return y, size


def rotate_tol(y, size, pos, inv_freq, interleaved, half_step):
    """|error| of a rotated element. Per unit of |x_a| + |x_b|: the turn held in
    fp32 (2^-25 half turns, pi 2^-25 < 2^-23 radians), sincospif (2 ulp, 2^-23),
    two products and a sum (2^-23 together): below 2^-21. The fixed-point
    fraction of a turn and the reference's own fp64 angle are off by at most
    2^-51 of the angle each. Then one rounding to the stored type."""
    n, d = y.shape[0], y.shape[-1]
    ang = np.abs(np.asarray(pos, np.float64))[:, None] * np.abs(np.asarray(inv_freq))[None]
    far = np.zeros((n, d))
    half = len(inv_freq)
    if interleaved:
        far[:, 0:2 * half:2] = far[:, 1:2 * half:2] = ang
    else:
        far[:, :half] = far[:, half:2 * half] = ang
    return size * (2.0 ** -21 + far[:, None] * 2.0 ** -50) + np.abs(y) * half_step + 2.0 ** -25


def attention(q, k_pool, v_pool, page_indptr, page_indices, seq_lens, q_indptr, group, *,
              scale=None, softcap=0.0, window=0, slopes=None, doc_starts=None, prefix_lens=None):
    """Rows of q over the paged cache. Returns dict(out, lse, dx, vmax, aw):
    dx bounds each row's fp32 logit error, vmax is the largest |v| seen and aw
    the softmax mean of |v| per dim."""
    S, d, n_phys = k_pool.shape[2], k_pool.shape[3], k_pool.shape[0]
    n, hq = q.shape[0], q.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    dx, vmax, aw = np.zeros((n, hq)), np.zeros((n, hq)), np.zeros((n, hq, d))
    eps = 2.0 ** -24
    for r in range(len(seq_lens)):
        L, e0, e1 = int(seq_lens[r]), int(page_indptr[r]), int(page_indptr[r + 1])
        a, b = int(q_indptr[r]), int(q_indptr[r + 1])
        held = min(L, (e1 - e0) * S)
        ids = np.asarray(page_indices[e0:e0 + -(-held // S)], np.int64)
        there = (ids >= 0) & (ids < n_phys)
        safe = np.where(there, ids, 0)
        j = np.arange(held)
        ok = np.repeat(there, S)[:held]
        for g in range(k_pool.shape[1]):
            k = k_pool[safe, g].reshape(-1, d)[:held].astype(np.float64)
            v = v_pool[safe, g].reshape(-1, d)[:held].astype(np.float64)
            for i in range(a, b):
                p = L - (b - a) + (i - a)
                hi = min(held, max(p + 1, int(prefix_lens[r]) if prefix_lens is not None else 0))
                lo = max(0, int(doc_starts[i]) if doc_starts is not None else 0)
                if window:
                    lo = max(lo, p - window + 1)
                see = ok & (j >= lo) & (j < hi)
                if not see.any():
                    continue
                kk, vv, jj = k[see], v[see], j[see]
                for h in range(g * group, (g + 1) * group):
                    qq = q[i, h].astype(np.float64)
                    x = scale * (kk @ qq)
                    # fp32 dot of d terms, the scale, and what follows it
                    err = (d + 4) * eps * scale * (np.abs(kk) @ np.abs(qq))
                    if softcap:
                        # tanh to 16 units of 2^-24 beside what its argument brings
                        err = err + 16 * eps * softcap
                        x = softcap * np.tanh(x / softcap)
                    if slopes is not None:
                        far = float(slopes[h]) * np.abs(p - jj)
                        x = x - far
                        err = err + 4 * eps * (np.abs(far) + np.abs(x))
                    m = x.max()
                    # in base 2, relative to the running maximum: two more roundings
                    near = x > m - 40
                    dx[i, h] = (err[near] + 6 * eps * (np.abs(x[near]) + abs(m) + 1)).max()
                    w = np.exp(x - m)
                    lse[i, h] = m + math.log(w.sum())
                    out[i, h] = w @ vv / w.sum()
                    aw[i, h] = w @ np.abs(vv) / w.sum()
                    vmax[i, h] = np.abs(vv).max()
    return dict(out=out, lse=lse, dx=dx, vmax=vmax, aw=aw)


def check_attention(out, lse, ref, half_step_p, half_step_out, n_keys):
    """out and lse against the fp64 form.

    A logit error of dx changes a weight by a factor within exp(+-dx) and so o
    by at most 2 dx aw per dim (dx < 1/4 here); ex2 adds 2^-21 relative to each
    weight. Rounding the weights (half_step_p relative; weights below the
    type's range lose at most 2^-24 of the largest each) and summing n_keys
    products in fp32 along a tree of tiles (n_keys / 16 + 64 roundings at most)
    come on top, then the output's own rounding."""
    out, lse = np.asarray(out, np.float64), np.asarray(lse, np.float64)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(out[empty] == 0)
    assert np.isfinite(out).all() and np.isfinite(lse[~empty]).all()
    dx = ref["dx"] + 2.0 ** -20
    assert dx.max() < 0.25
    sums = (n_keys / 16 + 64) * 2.0 ** -24
    rel = 2 * dx[..., None] + half_step_p + sums
    tol = rel * ref["aw"] + half_step_out * np.abs(ref["out"])
    if half_step_p:
        tol = tol + n_keys * 2.0 ** -24 * ref["vmax"][..., None] * 2.0 ** -6
    tol = tol + 2.0 ** -25
    err = np.abs(out - ref["out"])
    assert np.all(err <= tol), (float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))
    lt = dx + sums + 2.0 ** -22 * np.abs(np.where(empty, 0.0, ref["lse"]))
    le = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, ref["lse"]))
    assert np.all(le <= lt), float((le / lt).max())
