"""Cases, plain forms and exact values of normed appends and of the E4M3 cache.

Five operators belong together here. Models that norm every query and key head before the
position rotation write their cache through one pass (``norm_rope_append_kv``). The same pass
writes a cache of 8-bit floats (``quant_append_kv``), which the sparse layers read page by
selected page (``quant_sparse_decode_attn``), the dense layers as a whole
(``quant_dense_decode_attn``), and prompt attention after it has been read back into fp16 pages
(``quant_read_kv``).

The E4M3 cache keeps, for each page and KV head, one record of bytes: the codes of K
[d / 64][S][64], those of V [S / 16][d / 32][8][4][4][2][2] (dim 32 i + 4 g + c and token
16 s + 8 hi + 2 t + lo at [s][i][g][t][c][hi][lo]), the scales of K [S] and those of V [S]. A
scale is the exponent byte of a power of two; a code times its token's scale is the value.

``run`` computes the operators from elementary torch operations, or, where ``own`` is true,
through the package's calls.
"""

import math
import random

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
EPS = 1e-6


def _lens(text):
    return [int(x) for x in text.split(",")]


def _text(lens):
    return ",".join(str(int(x)) for x in lens)


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def _append(name, op, lens, before, **more):
    case = dict(op=op, lens=_text(lens), before=_text(before), h_kv=8, group=4, d=128, page=16, dtype="f16", fp8=False,
                norm=True, per_head=False, rotary=128, interleaved=False)
    case.update(more)
    return case if name is None else dict(name=name, **case)


def _read(name, lens, **more):
    case = dict(op="read", lens=_text(lens), h_kv=8, d=128, page=16)
    case.update(more)
    return case if name is None else dict(name=name, **case)


def _sparse(name, lens, k, **more):
    case = dict(op="sparse", lens=_text(lens), k=k, h_kv=8, group=4, d=128, page=16)
    case.update(more)
    return case if name is None else dict(name=name, **case)


def _dense(name, lens, **more):
    case = dict(op="dense", lens=_text(lens), h_kv=8, group=4, d=128, page=16, softcap=0.0, window=0, alibi=False, doc=0, prefix=0)
    case.update(more)
    return case if name is None else dict(name=name, **case)


def listed():
    r = random.Random(2004)
    ragged = [r.randint(8192, 131072) for _ in range(16)]
    r = random.Random(2007)
    served = [r.randint(1, 8192) for _ in range(63)] + [0]
    chunks, held = [517, 1, 0, 1023, 16, 33, 250], [0, 999, 64, 17, 15, 0, 4097]
    return [
        # one decode step of a batch into an fp16 cache: every request's new token; latency counts
        _append("norm_append_decode", "norm_append", [1] * 16, ragged),
        # chunks of several fp32 prompts, a weight for each head, half of a head rotated in interleaved pairs
        _append("norm_append_ragged_f32", "norm_append", chunks, held, h_kv=4, group=2, d=64, page=32, dtype="f32", per_head=True,
                rotary=32, interleaved=True),
        # a whole prompt with grouped heads into an fp16 cache with 8-bit summaries
        _append("norm_append_prompt", "norm_append", [65536], [0], fp8=True),
        # the decode step of that batch into the E4M3 cache
        _append("quant_append_decode", "quant_append", [1] * 16, ragged, fp8=True),
        # a long prompt into the E4M3 cache, one KV head per query head, keys that are not normed
        _append("quant_append_prompt_128k", "quant_append", [131072], [0], h_kv=32, group=1, page=32, norm=False),
        # short prompts of a batch read back, odd lengths, an empty request
        _read("read_ragged", [1777, 640, 0, 4095, 2, 1000], h_kv=4, d=64, page=32),
        # a long context read back for a chunk of its prompt
        _read("read_64k", [65536]),
        # one sparse layer's decode step: 128 of 2048 pages, one KV head per query head
        _sparse("sparse_llama_32k", [32768], 128, h_kv=32, group=1),
        # a batch of long ragged contexts, 256 pages each, and short ones with empty slots
        _sparse("sparse_gqa_batch", ragged[:14] + [2049, 31], 256),
        # the smallest call: one request, one head
        _dense("dense_tiny", [1000], h_kv=1, group=1, d=64),
        # a dense layer's decode step of a batch of long ragged contexts
        _dense("dense_gqa_ragged", ragged),
        # a serving batch of short and middling contexts: capped scores, a local window, packed documents
        _dense("dense_capped_window", served, h_kv=4, group=2, d=64, page=32, softcap=50.0, window=4096, alibi=True, doc=3000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_append", "quant_append", "read", "sparse", "sparse", "dense", "dense"])
    batch = _log(rng, 1, 32)
    h, G, d = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    common = dict(h_kv=h, d=d, page=rng.choice([16, 32]))
    if op in ("norm_append", "quant_append"):
        dtype = rng.choice(["f16", "f16", "f32"]) if op == "norm_append" else "f16"
        most = max(1, min(65536, 131072 * 96 * 64 // (batch * h * (G + 2) * d)))
        lens = [_log(rng, 1, most) if rng.random() < 0.9 else 0 for _ in range(batch)]
        lens[0] = max(lens[0], 1)
        return _append(None, op, lens, [rng.randint(0, 4096) for _ in lens], group=G, dtype=dtype,
                       fp8=dtype == "f16" and rng.random() < 0.5, norm=op == "norm_append" or rng.random() < 0.6,
                       per_head=rng.random() < 0.3, rotary=rng.choice([d, d // 2]), interleaved=rng.random() < 0.5, **common)
    most = max(1, min(131072, 8 * 131072 * 8 * 128 // (batch * h * d)))
    lens = [_log(rng, 1, most) if rng.random() < 0.95 else 0 for _ in range(batch)]
    lens[0] = max(lens[0], 1)
    if op == "read":
        return _read(None, lens, **common)
    if op == "sparse":
        return _sparse(None, lens, _log(rng, 1, 512), group=G, **common)
    return _dense(None, lens, group=G, softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                  alibi=rng.random() < 0.25, doc=rng.choice([0, 0, _log(rng, 16, 8192)]), prefix=rng.choice([0, 0, _log(rng, 1, 2048)]),
                  **common)


# ---------------------------------------------------------------------------------------------
# The E4M3 cache in torch
# ---------------------------------------------------------------------------------------------

def _record(S, d):
    return 2 * S * (d + 1)


def _k_order(x):
    """[..., S, d] in the order of a record's K codes."""
    S, d = x.shape[-2:]
    return x.unflatten(-1, (d // 64, 64)).transpose(-2, -3).reshape(*x.shape[:-2], S * d)


def _v_order(x):
    """[..., S, d] in the order of a record's V codes."""
    S, d = x.shape[-2:]
    n = x.dim() - 2
    x = x.unflatten(-1, (d // 32, 8, 4)).unflatten(n, (S // 16, 2, 4, 2))       # s hi t lo | i g c
    return x.permute(*range(n), n, n + 4, n + 5, n + 2, n + 6, n + 1, n + 3).reshape(*x.shape[:n], S * d)


def _k_rows(x, S, d):
    """The inverse of _k_order."""
    return x.unflatten(-1, (d // 64, S, 64)).transpose(-2, -3).flatten(-2)


def _v_rows(x, S, d):
    """The inverse of _v_order."""
    n = x.dim() - 1
    x = x.unflatten(-1, (S // 16, d // 32, 8, 4, 4, 2, 2))                      # s i g t c hi lo
    return x.permute(*range(n), n, n + 5, n + 3, n + 6, n + 1, n + 2, n + 4).flatten(-3).flatten(-5, -2)


def _quantise(x):
    """fp16 rows [..., d] -> E4M3 codes and the exponent e of each row."""
    x = x.float()
    top = x.abs().amax(dim=-1)
    m, p = torch.frexp(top)
    e = (p - 9 + (m > 0.875).to(p.dtype)).clamp(-14, 7)
    e = torch.where(top == 0, -14, e)
    return (x * torch.exp2(-e.float())[..., None]).to(E4M3), e


def _stored(codes, e):
    return codes.float() * torch.exp2(e.float())[..., None]


def _views(pool, S, d):
    """Codes and scales of K and of V, as floating tensors over the pool's bytes."""
    n = S * d
    return dict(k_codes=pool[..., :n].view(E4M3), v_codes=pool[..., n:2 * n].view(E4M3),
                k_scales=pool[..., 2 * n:2 * n + S].view(E8M0), v_scales=pool[..., 2 * n + S:].view(E8M0))


def _values(rec, S, d, dtype=torch.float32):
    """Records [..., R] -> the K and V that they hold, [..., S, d] each."""
    n = S * d
    scale = lambda b: torch.exp2(b.to(dtype) - 127.0)[..., None]  # noqa: E731
    k = _k_rows(rec[..., :n].view(E4M3), S, d).to(dtype).mul_(scale(rec[..., 2 * n:2 * n + S]))
    v = _v_rows(rec[..., n:2 * n].view(E4M3), S, d).to(dtype).mul_(scale(rec[..., 2 * n + S:]))
    return k, v


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _dtype(case):
    return torch.float16 if case.get("dtype", "f16") == "f16" else torch.float32


def _i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _random(g, dtype, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _pages(g, lens, page):
    """A page table over a pool whose pages are handed out in any order."""
    counts = [-(-n // page) for n in lens]
    indptr = np.concatenate([[0], np.cumsum(counts)])
    nnz = int(indptr[-1])
    n_phys = nnz + 5
    return dict(indptr=_i32(indptr), indices=torch.randperm(n_phys, generator=g, device="cuda")[:nnz].to(torch.int32),
                seq_lens=_i32(lens), nnz=nnz, n_phys=n_phys, most=max(counts + [1]))


def _quant_pool(g, n_phys, h, S, d):
    """A pool that holds something in every slot: values of unit size, a few channels of large keys."""
    pool = torch.empty((n_phys, h, _record(S, d)), dtype=torch.uint8, device="cuda")
    n = S * d
    large = torch.ones(d, device="cuda", dtype=torch.float16)
    large[torch.randperm(d, generator=g, device="cuda")[:4]] = 4
    step = max(1, (1 << 28) // (h * n))
    for a in range(0, n_phys, step):
        rec = pool[a:a + step]
        for at, order, by in ((0, _k_order, large), (1, _v_order, None)):
            x = _random(g, torch.float16, rec.shape[0], h, S, d)
            codes, e = _quantise(x if by is None else x.mul_(by))
            rec[..., at * n:(at + 1) * n] = order(codes.view(torch.uint8))
            rec[..., 2 * n + at * S:2 * n + (at + 1) * S] = (e + 127).to(torch.uint8)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, h, d, S = _dtype(case), case["h_kv"], case["d"], case["page"]
    hq = h * case.get("group", 1)
    lens = _lens(case["lens"])
    if "append" in case["op"]:
        before = _lens(case["before"])
        s = _pages(g, [a + b for a, b in zip(lens, before)], S)
        n = sum(lens)
        # queries, keys and values as one projection leaves them: three parts of each row
        qkv = _random(g, dt, n, (hq + 2 * h) * d)
        s.update(q=qkv[:, :hq * d].view(n, hq, d), k=qkv[:, hq * d:(hq + h) * d].view(n, h, d),
                 v=qkv[:, (hq + h) * d:].view(n, h, d),
                 append_indptr=_i32(np.concatenate([[0], np.cumsum(lens)])), before=_i32(before),
                 inv_freq=10000.0 ** (-torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64) / case["rotary"]),
                 q_out=torch.empty((n, hq, d), dtype=dt, device="cuda"), q_weight=None, k_weight=None)
        if case["norm"]:
            s["q_weight"] = 1 + 0.3 * _random(g, torch.float32, *((hq, d) if case["per_head"] else (d,)))
            s["k_weight"] = 1 + 0.3 * _random(g, torch.float32, *((h, d) if case["per_head"] else (d,)))
        # pages that hold earlier tokens have their summary; the others hold what was there before
        lo = _random(g, dt, s["n_phys"], h, d).abs_().neg_().sub_(2)
        hi = _random(g, dt, s["n_phys"], h, d).abs_().add_(2)
        s["summary"] = torch.stack([lo, hi], dim=2)
        if case["fp8"]:
            values = _e4m3_values()
            s["summary"] = torch.stack([_floor_e4m3(lo, values), _ceil_e4m3(hi, values)], dim=2)
        s["summary_out"] = s["summary"].view(E4M3) if case["fp8"] else s["summary"]
        if case["op"] == "norm_append":
            s["k_pool"], s["v_pool"] = (_random(g, dt, s["n_phys"], h, S, d) for _ in range(2))
        else:
            s["pool"] = _quant_pool(g, s["n_phys"], h, S, d)
            s["views"] = _views(s["pool"], S, d)
    else:
        s = _pages(g, lens, S)
        s["pool"] = _quant_pool(g, s["n_phys"], h, S, d)
        s["summary"] = torch.zeros((s["n_phys"], h, 2, d), dtype=dt, device="cuda")
        B = len(lens)
        if case["op"] == "read":
            s["k_pool"], s["v_pool"] = (_random(g, dt, s["nnz"] + 3, h, S, d) for _ in range(2))
            s["dst"] = torch.randperm(s["nnz"] + 3, generator=g, device="cuda")[:s["nnz"]].to(torch.int32)
        else:
            s.update(q=_random(g, dt, B, hq, d), out=torch.empty((B, hq, d), device="cuda"), lse=torch.empty((B, hq), device="cuda"))
        if case["op"] == "sparse":
            k, at, table = case["k"], s["indptr"].tolist(), s["indices"].long()
            sel = torch.full((B, h, k), -1, dtype=torch.int64, device="cuda")
            phys = sel.clone()
            for r, n in enumerate(-(-x // S) for x in lens):
                if n:
                    pick = torch.rand((h, n), generator=g, device="cuda")
                    pick[:, -1] = 2.0                                      # the page of the newest token is always of use
                    pick = pick.topk(min(k, n), dim=1).indices.sort(dim=1).values
                    sel[r, :, :pick.shape[1]] = pick
                    phys[r, :, :pick.shape[1]] = table[at[r] + pick]
            s["sel"], s["phys"] = sel.to(torch.int32), phys.to(torch.int32)
        if case["op"] == "dense":
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq) if case["alibi"] else None
            s["doc_starts"] = _i32([max(0, n - 1) // case["doc"] * case["doc"] for n in lens]) if case["doc"] else None
            s["prefix_lens"] = _i32([min(case["prefix"], n) for n in lens]) if case["prefix"] else None
    s["case"] = dict(case)
    if own:
        import query_aware_sparse_gb300 as qs
        s["table"] = qs.PageTable(s["indptr"], s["indices"], s["seq_lens"], nnz=s["nnz"])
        if "pool" in s:
            s["cache"] = qs.QuantCache(s["pool"], s["summary"], S, d)
        else:
            s["cache"] = qs.PagedCache(s["k_pool"], s["v_pool"], s["summary"])
        if "append" in case["op"]:
            s["norm"] = qs.QKNorm(s["q_weight"], s["k_weight"], EPS) if case["norm"] else None
        if case["op"] == "read":
            s["dst_cache"] = qs.PagedCache(s["k_pool"], s["v_pool"], torch.empty((s["nnz"] + 3, h, 2, d), dtype=dt, device="cuda"))
        if case["op"] == "dense":
            s["mods"] = qs.ScoreMods(softcap=case["softcap"], window=case["window"], alibi_slopes=s["slopes"],
                                     doc_starts=s["doc_starts"], prefix_lens=s["prefix_lens"])
        if case["op"] in ("sparse", "dense"):
            size = qs.quant_decode_workspace_size(len(lens), h, case["group"], d, S)
            s["workspace"] = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _e4m3_values():
    """All finite values of the 8-bit float, ascending, zero once."""
    codes = torch.arange(256, device="cuda", dtype=torch.uint8)
    codes = codes[(codes & 0x7f) != 0x7f]
    return torch.sort(codes[codes != 0x80].view(E4M3).float()).values


def _codes(values, at):
    return values[at.clamp(0, values.numel() - 1)].to(E4M3).view(torch.uint8)


def _floor_e4m3(x, values):
    return _codes(values, torch.searchsorted(values, x.float().contiguous(), right=True) - 1)


def _ceil_e4m3(x, values):
    return _codes(values, torch.searchsorted(values, x.float().contiguous()))


def _normed(x, weight):
    x = x.float()
    return x if weight is None else x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * weight


def _rotate(x, cos, sin, rotary, interleaved):
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., :rotary // 2], x[..., rotary // 2:rotary])
    c, e = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, e], dim=-1).flatten(-2) if interleaved else torch.cat([c, e], dim=-1)
    return torch.cat([turned, x[..., rotary:]], dim=-1)


def _plain_append(s):
    case, S, d, dt = s["case"], s["case"]["page"], s["case"]["d"], s["k"].dtype
    n, h = s["k"].shape[:2]
    row = torch.arange(n, device="cuda")
    r = torch.searchsorted(s["append_indptr"], row.to(torch.int32), right=True) - 1
    pos = s["before"][r] + row - s["append_indptr"][r]
    phys = s["indices"][(s["indptr"][r] + pos // S).long()].long()
    slot = (pos % S).long()
    angle = pos.double()[:, None] * s["inv_freq"][None, :]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q_out = _rotate(_normed(s["q"], s["q_weight"]), cos, sin, case["rotary"], case["interleaved"]).to(dt)
    k = _rotate(_normed(s["k"], s["k_weight"]), cos, sin, case["rotary"], case["interleaved"]).to(dt)
    pages, place = torch.unique(phys, return_inverse=True)
    if case["op"] == "norm_append":
        s["k_pool"][phys, :, slot] = k
        s["v_pool"][phys, :, slot] = s["v"]
        out = dict(k_pool=s["k_pool"], v_pool=s["v_pool"])
        k = k.float()
    else:
        # the touched pages as rows, the new tokens into them, and back
        m = S * d
        rec = s["pool"][pages]
        rows = [_k_rows(rec[..., :m], S, d), _v_rows(rec[..., m:2 * m], S, d)]
        (kc, ke), (vc, ve) = _quantise(k), _quantise(s["v"])
        k = _stored(kc, ke)
        for at, (code, e) in enumerate(((kc, ke), (vc, ve))):
            rows[at][place, :, slot] = code.view(torch.uint8)
            rec[place, :, 2 * m + at * S + slot] = (e + 127).to(torch.uint8)
        rec[..., :m], rec[..., m:2 * m] = _k_order(rows[0]), _v_order(rows[1])
        s["pool"][pages] = rec
        out = dict(s["views"])
    old = s["summary"][pages]
    old = old.view(E4M3).float() if case["fp8"] else old.float()
    lo, hi = old[:, :, 0].contiguous(), old[:, :, 1].contiguous()
    fresh = place[slot == 0]
    lo[fresh], hi[fresh] = math.inf, -math.inf
    lo.index_reduce_(0, place, k, "amin")
    hi.index_reduce_(0, place, k, "amax")
    if case["fp8"]:
        values = _e4m3_values()
        s["summary"][pages] = torch.stack([_floor_e4m3(lo, values), _ceil_e4m3(hi, values)], dim=2)
    else:
        s["summary"][pages] = torch.stack([lo, hi], dim=2).to(s["summary"].dtype)
    return dict(q=q_out, summary=s["summary_out"], **out)


def _plain_read(s):
    S, d = s["case"]["page"], s["case"]["d"]
    entry = torch.arange(s["nnz"], device="cuda")
    r = torch.searchsorted(s["indptr"], entry.to(torch.int32), right=True) - 1
    token = (entry - s["indptr"][r])[:, None] * S + torch.arange(S, device="cuda")
    held = (token < s["seq_lens"][r][:, None])[:, None, :, None]
    dst = s["dst"].long()
    for pool, x in zip((s["k_pool"], s["v_pool"]), _values(s["pool"][s["indices"].long()], S, d)):
        pool[dst] = torch.where(held, x.half(), pool[dst])
    return dict(k_pool=s["k_pool"], v_pool=s["v_pool"])


def _softmax(x, v):
    """x [..., G, keys] with -inf where hidden, v [..., keys, d] -> (out, lse)."""
    m = x.amax(dim=-1, keepdim=True).clamp_(min=-3e38)
    x.sub_(m).exp_()
    total = x.sum(dim=-1, keepdim=True)
    return torch.matmul(x, v) / total.clamp(min=1e-30), (m + total.log())[..., 0]


def _plain_attn(s):
    """Requests padded to the longest: [batch, h_kv, group, keys]."""
    case = s["case"]
    h, G, d, S = case["h_kv"], case["group"], case["d"], case["page"]
    lens, B = s["seq_lens"].long(), s["seq_lens"].shape[0]
    head = torch.arange(h, device="cuda")
    if case["op"] == "sparse":
        page = s["sel"].long()                                                       # [B, h, pages]
        rec = s["pool"][s["phys"].long().clamp(min=0), head[None, :, None]]
        held = page >= 0
    else:
        page = torch.arange(s["most"], device="cuda")[None].expand(B, -1)
        held = page * S < lens[:, None]
        ids = s["indices"].long()[torch.where(held, s["indptr"][:-1].long()[:, None] + page, 0)]
        rec = s["pool"][ids[:, None], head[None, :, None]]
        page, held = page[:, None], held[:, None]
    k, v = _values(rec, S, d)
    j = (page[..., None] * S + torch.arange(S, device="cuda")).flatten(-2)           # [B, h or 1, keys]
    hidden = ~held.repeat_interleave(S, dim=-1) | (j >= lens[:, None, None])
    x = torch.matmul(s["q"].float().view(B, h, G, d), k.flatten(2, 3).transpose(2, 3))
    x.mul_(1.0 / math.sqrt(d))
    if case["op"] == "dense":
        pos = (lens - 1)[:, None, None]
        hi = torch.maximum(pos + 1, s["prefix_lens"].long()[:, None, None]) if s["prefix_lens"] is not None else pos + 1
        hidden = hidden | (j >= hi)
        if case["window"]:
            hidden = hidden | (pos - j >= case["window"])
        if case["doc"]:
            hidden = hidden | (j < s["doc_starts"].long()[:, None, None])
        if case["softcap"]:
            x.div_(case["softcap"]).tanh_().mul_(case["softcap"])
        if case["alibi"]:
            x.addcmul_((pos - j).abs().float()[:, :, None], s["slopes"].view(1, h, G, 1), value=-1.0)
    x.masked_fill_(hidden[:, :, None], -math.inf)
    out, lse = _softmax(x, v.flatten(2, 3))
    return dict(out=out.view(B, h * G, d), lse=lse.view(B, h * G))


def run(state):
    s = state
    case = s["case"]
    if not own:
        return _plain_append(s) if "append" in case["op"] else _plain_read(s) if case["op"] == "read" else _plain_attn(s)
    import query_aware_sparse_gb300 as qs
    if case["op"] == "norm_append":
        qs.norm_rope_append_kv(s["cache"], s["table"], s["q"], s["k"], s["v"], s["append_indptr"], s["before"], s["norm"],
                               case["group"], inv_freq=s["inv_freq"], q_out=s["q_out"], interleaved=case["interleaved"])
        return dict(q=s["q_out"], k_pool=s["k_pool"], v_pool=s["v_pool"], summary=s["summary_out"])
    if case["op"] == "quant_append":
        qs.quant_append_kv(s["cache"], s["table"], s["q"], s["k"], s["v"], s["append_indptr"], s["before"], case["group"],
                           inv_freq=s["inv_freq"], norm=s["norm"], q_out=s["q_out"], interleaved=case["interleaved"])
        return dict(q=s["q_out"], summary=s["summary_out"], **s["views"])
    if case["op"] == "read":
        qs.quant_read_kv(s["cache"], s["table"], s["dst_cache"], dst_indices=s["dst"])
        return dict(k_pool=s["k_pool"], v_pool=s["v_pool"])
    if case["op"] == "sparse":
        out, lse = qs.quant_sparse_decode_attn(s["cache"], s["table"], s["q"], case["group"], s["sel"], s["phys"], case["k"],
                                               out=s["out"], lse=s["lse"], workspace=s["workspace"])
    else:
        out, lse = qs.quant_dense_decode_attn(s["cache"], s["table"], s["q"], case["group"], out=s["out"], lse=s["lse"],
                                              mods=s["mods"], workspace=s["workspace"])
    return dict(out=out, lse=lse)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def _visible(case):
    """Tokens that a query sees, and tokens of pages that hold one, over all requests."""
    S, tokens, held = case["page"], 0, 0
    for n in _lens(case["lens"]):
        if case["op"] == "sparse":
            pages = min(case["k"], -(-n // S))
            seen = 0 if n == 0 else (pages - 1) * S + n - (-(-n // S) - 1) * S       # the newest page is among them
            tokens, held = tokens + seen, held + seen
            continue
        lo, hi = 0, n
        if case["window"]:
            lo = max(lo, n - case["window"])
        if case["doc"]:
            lo = max(lo, max(0, n - 1) // case["doc"] * case["doc"])
        tokens += max(0, hi - lo)
        held += max(0, hi - lo)
    return tokens, held


def work(case):
    h, d, S = case["h_kv"], case["d"], case["page"]
    hq = h * case.get("group", 1)
    lens = _lens(case["lens"])
    if "append" in case["op"]:
        size = 2 if case["dtype"] == "f16" else 4
        before, n = _lens(case["before"]), sum(lens)
        pages = sum((b + a - 1) // S - b // S + 1 for a, b in zip(lens, before) if a)
        kept = sum(1 for a, b in zip(lens, before) if a and b % S)                   # pages whose summary is folded further
        summary = (pages + kept) * h * 2 * d * (1 if case["fp8"] else size)
        cache = 2 * h * (d * size if case["op"] == "norm_append" else d + 1)         # a token's K and V as they are kept
        return dict(bytes=n * ((2 * hq + 2 * h) * d * size + cache) + summary, flops=n * (hq + h) * (3 * case["rotary"] + 4 * d * case["norm"]))
    if case["op"] == "read":
        n = sum(lens)
        return dict(bytes=n * h * (2 * (d + 1) + 4 * d), flops=2 * n * h * d)
    seen, held = _visible(case)
    return dict(bytes=held * h * 2 * (d + 1) + len(lens) * hq * (6 * d + 4), flops=4 * seen * hq * d)


# ---------------------------------------------------------------------------------------------
# Exact values
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if "append" in case["op"] else _exact_read(case, s) if case["op"] == "read" else _exact_attn(case, s)


def _exact_append(case, s):
    """Pairs as complex numbers, turned by exp(i angle), request by request. What is kept in 8 bits: a code's value is
    compared with the real number that it rounds; scales, and boxes around rounded keys, have no value of their own."""
    S, rot = case["page"], case["rotary"]
    n, hq, d = s["q"].shape
    h, quant = case["h_kv"], case["op"] == "quant_append"
    q = torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
    if quant:
        m = S * d
        kp = _k_rows(s["pool"][..., :m], S, d).view(E4M3).double()
        vp = _v_rows(s["pool"][..., m:2 * m], S, d).view(E4M3).double()
    else:
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
    sm = None if case["fp8"] or quant else s["summary"].double()
    indptr, table = s["indptr"].tolist(), s["indices"].long()

    def turned(x, weight, pos):
        x = x.double()
        if weight is not None:
            x = x * weight.double() / torch.linalg.vector_norm(torch.nn.functional.pad(x, (0, 1), value=math.sqrt(EPS * d)), dim=-1,
                                                               keepdim=True) * math.sqrt(d)
        pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["interleaved"] else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        angle = (pos[:, None] * s["inv_freq"][None])[:, None]
        z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle)
        z = torch.view_as_real(z)
        x[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return x

    def scaled(x):
        """Over the power of two that a row's largest (fp16) element asks for."""
        top = x.abs().amax(dim=-1, keepdim=True).half().double()
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -40) / 448.0)).clamp(-14, 7)
        return x * 2.0 ** -e

    start = 0
    for r, (count, b) in enumerate(zip(_lens(case["lens"]), _lens(case["before"]))):
        at = 0
        while at < count:                                      # a page-aligned run of at most 16K tokens
            end = min(count, (b + at) // S * S + 16384 - b)
            rows = slice(start + at, start + end)
            pos = torch.arange(b + at, b + end, device="cuda")
            q[rows] = turned(s["q"][rows], s["q_weight"], pos.double())
            k = turned(s["k"][rows], s["k_weight"], pos.double())
            v = s["v"][rows].double()
            pages = table[indptr[r]:][pos // S]
            kp[pages, :, pos % S] = scaled(k) if quant else k
            vp[pages, :, pos % S] = scaled(v) if quant else v
            if sm is not None:
                lp0, lp1 = (b + at) // S, (b + end - 1) // S
                pad = torch.full(((lp1 - lp0 + 1) * S, h, d), math.nan, dtype=torch.float64, device="cuda")
                pad[pos - lp0 * S] = k
                pad = pad.view(-1, S, h, d)
                none = pad.isnan()
                lo = pad.masked_fill(none, math.inf).amin(1)
                hi = pad.masked_fill(none, -math.inf).amax(1)
                ids = table[indptr[r] + lp0: indptr[r] + lp1 + 1]
                if (b + at) % S:                               # the first page held tokens before
                    lo[0] = torch.minimum(lo[0], sm[ids[0], :, 0])
                    hi[0] = torch.maximum(hi[0], sm[ids[0], :, 1])
                sm[ids, :, 0], sm[ids, :, 1] = lo, hi
            at = end
        start += count
    if quant:
        return dict(q=q, k_codes=_k_order(kp), v_codes=_v_order(vp), k_scales=None, v_scales=None, summary=None)
    return dict(q=q, k_pool=kp, v_pool=vp, summary=sm)


def _e4m3_exact(code):
    """An E4M3 code's value in 64 bits, from its bits."""
    c = code.to(torch.int64)
    e, m = c >> 3 & 15, c & 7
    x = torch.where(e == 0, m.double() * 2.0 ** -9, (8 + m).double() * torch.exp2(e.double() - 10))
    return torch.where(c >= 128, -x, x)


def _exact_rows(rec, at, S, d):
    """K (at 0) or V (at 1) of records [n, R], token by token: [n, S, d]."""
    m = S * d
    token, dim = torch.meshgrid(torch.arange(S, device="cuda"), torch.arange(d, device="cuda"), indexing="ij")
    if at == 0:
        place = dim // 64 * (64 * S) + token * 64 + dim % 64
    else:
        lane = dim % 32 // 4 * 4 + token % 8 // 2
        place = (((token // 16 * (d // 32) + dim // 32) * 32 + lane) * 4 + dim % 4) * 4 + token % 16 // 8 * 2 + token % 2
    codes = rec[:, at * m + place.flatten()].view(-1, S, d)
    return _e4m3_exact(codes) * torch.exp2(rec[:, 2 * m + at * S:2 * m + (at + 1) * S].double() - 127)[..., None]


def _exact_read(case, s):
    S, d = case["page"], case["d"]
    out = [s["k_pool"].double(), s["v_pool"].double()]
    indptr = s["indptr"].tolist()
    for r, n in enumerate(_lens(case["lens"])):
        for a in range(indptr[r], indptr[r + 1], 1024):
            b = min(indptr[r + 1], a + 1024)
            ids, dst = s["indices"][a:b].long(), s["dst"][a:b].long()
            left = n - (a - indptr[r]) * S
            for head in range(case["h_kv"]):
                for at in (0, 1):
                    rows = _exact_rows(s["pool"][ids, head], at, S, d)
                    there = torch.arange(rows.shape[0] * S, device="cuda") < left
                    flat = out[at][dst, head].reshape(-1, d)
                    flat[there] = rows.reshape(-1, d)[there]
                    out[at][dst, head] = flat.view(-1, S, d)
    return dict(k_pool=out[0], v_pool=out[1])


def _exact_attn(case, s):
    h, G, d, S = case["h_kv"], case["group"], case["d"], case["page"]
    lens = _lens(case["lens"])
    out = torch.zeros((len(lens), h * G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), h * G), -math.inf, dtype=torch.float64, device="cuda")
    indptr = s["indptr"].tolist()
    for r, L in enumerate(lens):
        pos = L - 1
        lo, hi = 0, L
        if case["op"] == "dense":
            lo = max(0, pos - case["window"] + 1) if case["window"] else 0
            lo = max(lo, pos // case["doc"] * case["doc"]) if case["doc"] and L else lo
        if hi <= lo:
            continue
        for g in range(h):
            if case["op"] == "sparse":
                page = s["sel"][r, g].long()
                page = page[page >= 0]
            else:
                page = torch.arange(lo // S, -(-hi // S), device="cuda")
            rec = s["pool"][s["indices"].long()[indptr[r] + page], g]
            j = (page[:, None] * S + torch.arange(S, device="cuda")).flatten()
            see = (j >= lo) & (j < hi)
            k, v = (_exact_rows(rec, at, S, d).reshape(-1, d)[see] for at in (0, 1))
            j = j[see]
            t = s["q"][r, g * G:(g + 1) * G].double() @ k.T / math.sqrt(d)
            if case["op"] == "dense":
                if case["softcap"]:
                    t = case["softcap"] * torch.tanh(t / case["softcap"])
                if case["alibi"]:
                    t = t - s["slopes"][g * G:(g + 1) * G].double()[:, None] * (pos - j).abs()
            lse[r, g * G:(g + 1) * G] = torch.logsumexp(t, dim=1)
            out[r, g * G:(g + 1) * G] = torch.softmax(t, dim=1) @ v
    return dict(out=out, lse=lse)
