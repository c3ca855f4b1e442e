"""Cases, plain forms and exact values of the dense-layer operators around the paged cache.

Three operators belong together here. A layer that attends densely (the first layers of a
model that selects pages elsewhere, and every layer while its prompt is read in) rotates its
queries and keys and puts keys and values into their pages (``rope_append_kv``), attends with
all of a prompt chunk's queries over the cache (``prefill_attn``), and then with one new query
per request (``dense_decode_attn``).

``run`` computes them from elementary torch operations, or, where ``own`` is true, through the
package's calls.
"""

import math
import random

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn


def _lens(text):
    return [int(x) for x in text.split(",")]


def _text(lens):
    return ",".join(str(int(x)) for x in lens)


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def _append(name, lens, before, **more):
    case = dict(op="append", lens=_text(lens), before=_text(before), h_kv=8, group=4, d=128, page=16,
                dtype="f16", fp8=False, rotary=128, interleaved=False)
    case.update(more)
    return case if name is None else dict(name=name, **case)


def _decode(name, lens, **more):
    case = dict(op="decode", lens=_text(lens), h_kv=8, group=4, d=128, page=16, dtype="f16",
                softcap=0.0, window=0, alibi=False, doc=0)
    case.update(more)
    return case if name is None else dict(name=name, **case)


def _prefill(name, lens, rows, **more):
    case = dict(op="prefill", lens=_text(lens), rows=_text(rows), h_kv=8, group=4, d=128, page=16,
                dtype="f16", softcap=0.0, window=0, alibi=False, doc=0, prefix=0)
    case.update(more)
    return case if name is None else dict(name=name, **case)


def listed():
    r = random.Random(1004)
    ragged = [r.randint(8192, 131072) for _ in range(16)]
    r = random.Random(1007)
    served = [r.randint(1, 8192) for _ in range(64)]
    drafts = [r.randint(2, 32768) for _ in range(16)]
    return [
        # one decode step of a batch: every request's new token, fp8 summaries; latency counts
        _append("append_decode_e4m3", [1] * 16, ragged, fp8=True),
        # chunks of several prompts in one batch, half of each head rotated in interleaved pairs
        _append("append_ragged_f32", [517, 1, 0, 1023, 16, 33, 250], [0, 999, 64, 17, 15, 0, 4097], h_kv=4, group=2, d=64,
                page=32, dtype="f32", rotary=32, interleaved=True),
        # a whole long prompt of one request
        _append("append_prompt_128k", [131072], [0], h_kv=32, group=1, page=32),
        # the smallest call: one request, one head, fp32
        _decode("decode_tiny_f32", [1000], h_kv=1, group=1, d=64, dtype="f32"),
        # a dense layer's decode step over a 32K context, one KV head per query head
        _decode("decode_llama_32k", [32768], h_kv=32, group=1),
        # a batch of long ragged contexts, grouped heads, pages in any order
        _decode("decode_gqa_ragged", ragged),
        # a serving batch of short and middling contexts: capped scores in a local window
        _decode("decode_capped_window", served, h_kv=4, group=2, d=64, page=32, softcap=50.0, window=4096),
        # a prompt of 16K tokens, every query head with its own KV head
        _prefill("prefill_llama_16k", [16384], [16384], h_kv=32, group=1),
        # a chunk of a long prompt over what is cached already, capped scores
        _prefill("prefill_chunk_capped", [65536], [2048], softcap=50.0),
        # packed documents of several requests, distance bias, odd sizes
        _prefill("prefill_documents_alibi", [1777, 640, 4095, 2, 1000], [1777, 129, 2047, 1, 0], h_kv=4, group=8, d=64, page=32,
                 alibi=True, doc=700),
        # a few drafted tokens per request, checked against long caches
        _prefill("prefill_draft_check", drafts, [min(4, n) for n in drafts]),
        # fp32: a prompt whose first part attends in both directions
        _prefill("prefill_prefix_f32", [1000], [1000], h_kv=2, group=2, d=64, dtype="f32", prefix=300, window=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "prefill"])
    common = dict(h_kv=rng.choice([1, 2, 4, 8, 16, 32]), group=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                  page=rng.choice([16, 32]), dtype=rng.choice(["f16", "f16", "f16", "f32"]))
    heads = common["h_kv"] * common["group"]
    batch = _log(rng, 1, 32)
    if op == "append":
        most = max(1, min(65536, 131072 * 96 * 64 // (batch * (heads + 2 * common["h_kv"]) * common["d"])))
        lens = [_log(rng, 1, most) for _ in range(batch)]
        return _append(None, lens, [rng.randint(0, 4096) for _ in lens], fp8=common["dtype"] == "f16" and rng.random() < 0.5,
                       rotary=rng.choice([common["d"], common["d"] // 2]), interleaved=rng.random() < 0.5, **common)
    mods = dict(softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, 8192)]), alibi=rng.random() < 0.25,
                doc=rng.choice([0, 0, _log(rng, 16, 8192)]))
    if op == "decode":
        most = max(1, min(131072, 16 * 131072 * 8 * 128 // (batch * common["h_kv"] * common["d"])))
        return _decode(None, [_log(rng, 1, most) for _ in range(batch)], **common, **mods)
    if common["dtype"] == "f32":
        common["h_kv"], heads = min(common["h_kv"], 4), min(common["h_kv"], 4) * common["group"]
    rows = _log(rng, 1, 8192)
    most = max(rows, min(65536, 32 * 8192 * 8192 // (batch * heads * rows), 16 * 131072 * 8 * 128 // (batch * common["h_kv"] * common["d"])))
    if batch * heads * rows * most > 32 * 8192 * 8192:
        batch = max(1, 32 * 8192 * 8192 // (heads * rows * most))
        rows = max(1, min(rows, 32 * 8192 * 8192 // (batch * heads * most)))
    lens = [_log(rng, rows, most) for _ in range(batch)]
    return _prefill(None, lens, [rng.randint(1, rows) for _ in lens], prefix=rng.choice([0, 0, _log(rng, 1, 2048)]), **common, **mods)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _dtype(case):
    return torch.float16 if case["dtype"] == "f16" else torch.float32


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, h, d, S = _dtype(case), case["h_kv"], case["d"], case["page"]
    hq = h * case["group"]
    lens = _lens(case["lens"])
    if case["op"] == "append":
        before = _lens(case["before"])
        s = _pages(g, [a + b for a, b in zip(lens, before)], S)
        n = sum(lens)
        # queries, keys and values as one projection leaves them: three parts of each row
        qkv = _random(g, dt, n, (hq + 2 * h) * d)
        s.update(q=qkv[:, :hq * d].view(n, hq, d), k=qkv[:, hq * d:(hq + h) * d].view(n, h, d),
                 v=qkv[:, (hq + h) * d:].view(n, h, d),
                 append_indptr=_i32(np.concatenate([[0], np.cumsum(lens)])), before=_i32(before),
                 inv_freq=10000.0 ** (-torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64) / case["rotary"]))
        # pages that hold earlier tokens have their summary; the others hold what was there before
        lo = _random(g, dt, s["n_phys"], h, d).abs_().neg_().sub_(2)
        hi = _random(g, dt, s["n_phys"], h, d).abs_().add_(2)
        summary = torch.stack([lo, hi], dim=2)
        if case["fp8"]:
            values = _e4m3_values()
            summary = torch.stack([_floor_e4m3(lo, values), _ceil_e4m3(hi, values)], dim=2)
        s["q_out"] = torch.empty((n, hq, d), dtype=dt, device="cuda")
    else:
        s = _pages(g, lens, S)
        rows = _lens(case["rows"]) if case["op"] == "prefill" else [1] * len(lens)
        starts = np.concatenate([[0], np.cumsum(rows)])
        n = int(starts[-1])
        s.update(q=_random(g, dt, n, hq, d), q_indptr=_i32(starts), n_q=n, most_rows=max(rows),
                 out=torch.empty((n, hq, d), dtype=dt if case["op"] == "prefill" else torch.float32, device="cuda"),
                 lse=torch.empty((n, hq), device="cuda"))
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq) if case["alibi"] else None
        at = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, rows)]) if n else np.zeros(0)
        s["doc_starts"] = _i32(at // case["doc"] * case["doc"]) if case["doc"] else None
        s["prefix_lens"] = _i32([min(case["prefix"], a) for a in lens]) if case.get("prefix") else None
        summary = torch.zeros((s["n_phys"], h, 2, d), dtype=dt, device="cuda")
    k_pool = _random(g, dt, s["n_phys"], h, S, d)
    if case["op"] != "append":
        k_pool[..., torch.randperm(d, generator=g, device="cuda")[:4]] *= 4   # a few channels of large keys
    s.update(case=dict(case), k_pool=k_pool, v_pool=_random(g, dt, s["n_phys"], h, S, d), summary=summary)
    if own:
        import query_aware_sparse_gb300 as qs
        s["cache"] = qs.PagedCache(s["k_pool"], s["v_pool"], s["summary"])
        s["table"] = qs.PageTable(s["indptr"], s["indices"], s["seq_lens"], nnz=s["nnz"])
        if case["op"] != "append":
            s["mods"] = qs.ScoreMods(softcap=case["softcap"], window=case["window"], alibi_slopes=s["slopes"],
                                     doc_starts=s["doc_starts"], prefix_lens=s["prefix_lens"])
            size = (qs.prefill_workspace_size(len(lens), n, s["nnz"], h, case["group"], d, S, dt) if case["op"] == "prefill" else
                    qs.dense_decode_workspace_size(len(lens), s["nnz"], h, case["group"], d, S, dt))
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


def _rotate(x, cos, sin, rotary, interleaved):
    x = x.float()
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., :rotary // 2], x[..., rotary // 2:rotary])
    c, e = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, e], dim=-1).flatten(-2) if interleaved else torch.cat([c, e], dim=-1)
    return torch.cat([turned, x[..., rotary:]], dim=-1)


def _plain_append(s):
    case, S = s["case"], s["case"]["page"]
    n = s["k"].shape[0]
    row = torch.arange(n, device="cuda")
    r = torch.searchsorted(s["append_indptr"], row.to(torch.int32), right=True) - 1
    pos = s["before"][r] + row - s["append_indptr"][r]
    phys = s["indices"][(s["indptr"][r] + pos // S).long()].long()
    slot = (pos % S).long()
    angle = pos.double()[:, None] * s["inv_freq"][None, :]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q_out = _rotate(s["q"], cos, sin, case["rotary"], case["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, case["rotary"], case["interleaved"]).to(s["k"].dtype)
    s["k_pool"][phys, :, slot] = k
    s["v_pool"][phys, :, slot] = s["v"]
    pages, place = torch.unique(phys, return_inverse=True)
    old = s["summary"][pages]
    old = old.view(E4M3).float() if case["fp8"] else old.float()
    lo, hi = old[:, :, 0].contiguous(), old[:, :, 1].contiguous()
    fresh = place[slot == 0]
    lo[fresh], hi[fresh] = math.inf, -math.inf
    lo.index_reduce_(0, place, k.float(), "amin")
    hi.index_reduce_(0, place, k.float(), "amax")
    if case["fp8"]:
        values = _e4m3_values()
        s["summary"][pages] = torch.stack([_floor_e4m3(lo, values), _ceil_e4m3(hi, values)], dim=2)
    else:
        s["summary"][pages] = torch.stack([lo, hi], dim=2).to(s["summary"].dtype)
    return dict(q=q_out, k_pool=s["k_pool"], v_pool=s["v_pool"], summary=s["summary"].view(E4M3) if case["fp8"] else s["summary"])


def _plain_attn(s):
    """Requests padded to the longest: [batch, h_kv, group * rows, keys]."""
    case = s["case"]
    h, G, d, S = case["h_kv"], case["group"], case["d"], case["page"]
    lens, B = s["seq_lens"].long(), s["seq_lens"].shape[0]
    first, rows, R = s["q_indptr"][:-1].long(), (s["q_indptr"][1:] - s["q_indptr"][:-1]).long(), s["most_rows"]
    page = torch.arange(s["most"], device="cuda")
    held = page[None] * S < lens[:, None]
    ids = s["indices"].long()[torch.where(held, s["indptr"][:-1].long()[:, None] + page[None], 0)]
    j = torch.arange(s["most"] * S, device="cuda")
    i = torch.arange(R, device="cuda")
    there = i[None] < rows[:, None]
    at = torch.where(there, first[:, None] + i[None], 0)
    pos = lens[:, None] - rows[:, None] + i[None]
    hi = torch.minimum(lens[:, None], torch.maximum(pos + 1, s["prefix_lens"].long()[:, None]) if s["prefix_lens"] is not None else pos + 1)
    lo = pos - case["window"] + 1 if case["window"] else torch.zeros_like(pos)
    lo = torch.maximum(lo, s["doc_starts"].long()[at]) if s["doc_starts"] is not None else lo
    hidden = (j < lo[..., None]) | (j >= hi[..., None])                              # [B, R, keys]
    q = s["q"][at].float().view(B, R, h, G, d).permute(0, 2, 3, 1, 4).reshape(B, h, G * R, d)
    k = s["k_pool"][ids].float().transpose(1, 2).reshape(B, h, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, h, G, R, -1)
    del k
    x.mul_(1.0 / math.sqrt(d))
    if case["softcap"]:
        x.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    if case["alibi"]:
        far = (pos[..., None] - j).abs().float()[:, None, None]
        x.addcmul_(far, s["slopes"].view(1, h, G, 1, 1), value=-1.0)
    x.masked_fill_(hidden[:, None, None], -math.inf)
    m = x.amax(dim=-1, keepdim=True).clamp_(min=-3e38)
    x.sub_(m).exp_()
    total = x.sum(dim=-1, keepdim=True)
    v = s["v_pool"][ids].float().transpose(1, 2).reshape(B, h, -1, d)
    v.masked_fill_((j >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x.view(B, h, G * R, -1), v).view(B, h, G, R, d) / total.clamp(min=1e-30)
    lse = (m + total.log())[..., 0]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, R, h * G, d)[there]
    return dict(out=out.to(s["out"].dtype), lse=lse.permute(0, 3, 1, 2).reshape(B, R, h * G)[there])


def run(state):
    s = state
    case = s["case"]
    if not own:
        return _plain_append(s) if case["op"] == "append" else _plain_attn(s)
    import query_aware_sparse_gb300 as qs
    if case["op"] == "append":
        qs.rope_append_kv(s["cache"], s["table"], s["q"], s["k"], s["v"], s["append_indptr"], s["before"], s["inv_freq"],
                          case["group"], q_out=s["q_out"], interleaved=case["interleaved"])
        return dict(q=s["q_out"], k_pool=s["k_pool"], v_pool=s["v_pool"], summary=s["summary"].view(E4M3) if case["fp8"] else s["summary"])
    if case["op"] == "decode":
        out, lse = qs.dense_decode_attn(s["cache"], s["table"], s["q"], case["group"], out=s["out"], lse=s["lse"], mods=s["mods"],
                                        workspace=s["workspace"])
    else:
        out, lse = qs.prefill_attn(s["cache"], s["table"], s["q"], case["group"], s["q_indptr"], out=s["out"], lse=s["lse"],
                                   mods=s["mods"], workspace=s["workspace"])
    return dict(out=out, lse=lse)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def _visible(case):
    """(query, key) pairs of one head, and (request, page) pairs that some query reads."""
    pairs, pages, S = 0, 0, case["page"]
    lens = _lens(case["lens"])
    for n, rows in zip(lens, _lens(case["rows"]) if case["op"] == "prefill" else [1] * len(lens)):
        pos = np.arange(n - rows, n, dtype=np.int64)
        lo, hi = np.zeros_like(pos), np.minimum(n, np.maximum(pos + 1, min(case.get("prefix", 0), n)))
        if case["window"]:
            lo = np.maximum(lo, pos - case["window"] + 1)
        if case["doc"]:
            lo = np.maximum(lo, pos // case["doc"] * case["doc"])
        hi = np.maximum(lo, hi)
        pairs += int((hi - lo).sum())
        if rows and (hi > lo).any():
            pages += int(-(-hi.max() // S) - lo[hi > lo].min() // S)
    return pairs, pages


def work(case):
    size = 2 if case["dtype"] == "f16" else 4
    h, d, S = case["h_kv"], case["d"], case["page"]
    hq = h * case["group"]
    if case["op"] == "append":
        lens, before = _lens(case["lens"]), _lens(case["before"])
        n = sum(lens)
        pages = sum((b + a - 1) // S - b // S + 1 for a, b in zip(lens, before) if a)
        kept = sum(1 for a, b in zip(lens, before) if a and b % S)         # pages whose summary is folded further
        summary = (pages + kept) * h * 2 * d * (1 if case["fp8"] else size)
        return dict(bytes=2 * n * (hq + 2 * h) * d * size + summary, flops=3 * n * (hq + h) * case["rotary"])
    pairs, pages = _visible(case)
    n = sum(_lens(case["rows"])) if case["op"] == "prefill" else len(_lens(case["lens"]))
    out = size if case["op"] == "prefill" else 4
    return dict(bytes=pages * S * h * d * 2 * size + n * hq * (d * (size + out) + 4), flops=4 * pairs * hq * d)


# ---------------------------------------------------------------------------------------------
# Exact values
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attn(case, s)


def _exact_append(case, s):
    """Pairs as complex numbers, turned by exp(i angle), request by request."""
    S, rot = case["page"], case["rotary"]
    n, hq, d = s["q"].shape
    h = case["h_kv"]
    q = torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    sm = None if case["fp8"] else s["summary"].double()
    indptr, table = s["indptr"].tolist(), s["indices"].long()

    def turned(x, pos):
        x = x.double()
        pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["interleaved"] else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        angle = (pos[:, None] * s["inv_freq"][None])[:, None]
        z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle)
        z = torch.view_as_real(z)
        x[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return x

    start = 0
    for r, (count, b) in enumerate(zip(_lens(case["lens"]), _lens(case["before"]))):
        at = 0
        while at < count:                                      # a page-aligned run of at most 16K tokens
            end = min(count, (b + at) // S * S + 16384 - b)
            rows = slice(start + at, start + end)
            pos = torch.arange(b + at, b + end, device="cuda")
            q[rows] = turned(s["q"][rows], pos.double())
            k = turned(s["k"][rows], pos.double())
            pages = table[indptr[r]:][pos // S]
            kp[pages, :, pos % S] = k
            vp[pages, :, pos % S] = s["v"][rows].double()
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
    return dict(q=q, k_pool=kp, v_pool=vp, summary=sm)


def _exact_attn(case, s):
    h, G, d, S = case["h_kv"], case["group"], case["d"], case["page"]
    n = s["n_q"]
    out = torch.zeros((n, h * G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n, h * G), -math.inf, dtype=torch.float64, device="cuda")
    indptr, starts = s["indptr"].tolist(), s["q_indptr"].tolist()
    for r, L in enumerate(_lens(case["lens"])):
        a, b = starts[r], starts[r + 1]
        ids = s["indices"][indptr[r]:indptr[r] + -(-L // S)].long()
        k_all, v_all = s["k_pool"][ids], s["v_pool"][ids]
        j = torch.arange(L, device="cuda")
        for c in range(a, b, 4096):                            # rows of one request, 4096 at a time
            e = min(b, c + 4096)
            pos = torch.arange(c, e, device="cuda") - a + L - (b - a)
            end = pos + 1
            if s["prefix_lens"] is not None:
                end = end.clamp(min=int(s["prefix_lens"][r]))
            seen = j[None] < end.clamp(max=L)[:, None]
            if case["window"]:
                seen &= pos[:, None] - j[None] < case["window"]
            if case["doc"]:
                seen &= j[None] >= s["doc_starts"][c:e].long()[:, None]
            first = int(seen.any(0).int().argmax()) if bool(seen.any()) else 0
            last = int(end.clamp(max=L).max())
            if last <= first:
                continue
            jj, see = j[first:last], seen[:, first:last]
            for g in range(h):
                k = k_all[:, g].reshape(-1, d)[first:last].double()
                v = v_all[:, g].reshape(-1, d)[first:last].double()
                for x in range(g * G, (g + 1) * G):
                    t = (s["q"][c:e, x].double() @ k.T) / math.sqrt(d)
                    if case["softcap"]:
                        t = case["softcap"] * torch.tanh(t / case["softcap"])
                    if case["alibi"]:
                        t -= s["slopes"][x].double() * (pos[:, None] - jj[None]).abs()
                    t = torch.where(see, t, -math.inf)
                    z = torch.logsumexp(t, dim=1)
                    lse[c:e, x] = z
                    p = torch.exp(t - torch.where(torch.isinf(z), 0.0, z)[:, None])
                    out[c:e, x] = p @ v
    return dict(out=out, lse=lse)
