"""query_aware_sparse_gb300 — Quest-style query-aware page selection on GB300.

A thin Python binding over ``libquest.so`` (the C ABI in ``include/quest.h``).
Every function here only marshals arguments (tensor data pointers, sizes and
the current CUDA stream) and calls the library; all the computation runs in
the library's CUDA kernels. There is no fallback: if the library is missing or
a call fails, an exception is raised.

Tensors are torch tensors on the current CUDA device (torch is used for device
memory and streams only).
"""

from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libquest.so")

QUEST_F32, QUEST_F16 = 0, 1
DEVERR = {1: "page id outside the pool", 2: "beyond the page table",
          4: "selected page holds no valid token", 8: "in-kernel wait timed out",
          16: "key beyond +-448 under an E4M3 summary, or a number that an E4M3 cache cannot hold"}


class QuestCache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("summary", ctypes.c_void_p), ("n_phys", ctypes.c_int32),
                ("h_kv", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("summary_fp8", ctypes.c_int32)]


class QuestPages(ctypes.Structure):
    _fields_ = [("page_indptr", ctypes.c_void_p), ("page_indices", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("nnz", ctypes.c_int32)]


class QuestRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class QuestScoreMods(ctypes.Structure):
    _fields_ = [("alibi_slopes", ctypes.c_void_p), ("doc_starts", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p), ("softcap", ctypes.c_float),
                ("window", ctypes.c_int32)]


class QuestQKNorm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("q_per_head", ctypes.c_int32), ("k_per_head", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class QuestQuantCache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("summary", ctypes.c_void_p),
                ("n_phys", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("summary_fp8", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libquest.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m query_aware_sparse_gb300.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.quest_append_kv.argtypes = [P, P, P, P, I32, P, P, P]
        L.quest_score_pages.argtypes = [P, P, P, I32, P, P]
        L.quest_score_pages_per_head.argtypes = [P, P, P, I32, P, P]
        L.quest_union_decode_attn.argtypes = [P, P, P, I32, P, I32, P, P, ctypes.c_float, P, P,
                                              P, P, SZ, P]
        L.quest_union_decode_attn.restype = I32
        L.quest_union_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32, I32]
        L.quest_union_workspace_size.restype = SZ
        L.quest_select_topk.argtypes = [P, I32, I32, P, I32, I32, I32, P, P, P, P]
        L.quest_sparse_decode_attn.argtypes = [P, P, P, I32, P, P, I32, P, P,
                                               ctypes.c_float, P, SZ, P]
        L.quest_sparse_decode_attn_noalloc.argtypes = [P, P, P, I32, P, P, I32, P, P,
                                                       ctypes.c_float, P]
        L.quest_sparse_decode_attn_noalloc.restype = I32
        L.quest_attn_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32]
        L.quest_attn_workspace_size.restype = SZ
        L.quest_decode_step.argtypes = [P, P, P, P, P, I32, I32, I32, I32, P, P, P, P, P, P,
                                        ctypes.c_float, P, SZ, P]
        L.quest_decode_step.restype = I32
        L.quest_decode_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32, I32, I32]
        L.quest_decode_workspace_size.restype = SZ
        L.quest_decode_step_kernel.argtypes = [I32, I32, I32, I32, I32, I32, I32, I32]
        L.quest_decode_step_kernel.restype = I32
        L.quest_recall_diagnostics.argtypes = [P, P, P, I32, P, I32, I32, ctypes.c_float, P, P,
                                               P, P, P, SZ, P]
        L.quest_recall_diagnostics.restype = I32
        L.quest_diag_workspace_size.argtypes = [I32, I32, I32, I32]
        L.quest_diag_workspace_size.restype = SZ
        I64 = ctypes.c_int64
        L.quest_rope_append_kv.argtypes = [P, P, P, P, P, P, I64, I64, I64, I32, I32, P, P, P, P]
        L.quest_rope_append_kv.restype = I32
        L.quest_dense_decode_attn.argtypes = [P, P, P, I32, P, P, P, ctypes.c_float, P, SZ, P]
        L.quest_dense_decode_attn.restype = I32
        L.quest_dense_decode_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32, I32]
        L.quest_dense_decode_workspace_size.restype = SZ
        L.quest_prefill_attn.argtypes = [P, P, P, I32, P, I32, P, P, P, ctypes.c_float, P, SZ, P]
        L.quest_prefill_attn.restype = I32
        L.quest_prefill_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32, I32, I32]
        L.quest_prefill_workspace_size.restype = SZ
        append = [P, P, P, P, P, P, P, I64, I64, I64, I32, I32, P, P, P, P]
        L.quest_norm_rope_append_kv.argtypes = L.quest_quant_append_kv.argtypes = append
        L.quest_norm_rope_append_kv.restype = L.quest_quant_append_kv.restype = I32
        L.quest_quant_page_bytes.argtypes = [I32, I32]
        L.quest_quant_page_bytes.restype = SZ
        L.quest_quant_read_kv.argtypes = [P, P, P, P, I32, P, P]
        L.quest_quant_read_kv.restype = I32
        L.quest_quant_sparse_decode_attn.argtypes = [P, P, P, I32, P, P, I32, P, P, ctypes.c_float,
                                                     P, SZ, P]
        L.quest_quant_sparse_decode_attn.restype = I32
        L.quest_quant_dense_decode_attn.argtypes = [P, P, P, I32, P, P, P, ctypes.c_float, P, SZ, P]
        L.quest_quant_dense_decode_attn.restype = I32
        L.quest_quant_decode_workspace_size.argtypes = [I32, I32, I32, I32, I32]
        L.quest_quant_decode_workspace_size.restype = SZ
        L.quest_set_trace.argtypes = [P, I32, I32, I32, I32, I32, I32, I32, I32]
        L.quest_set_trace.restype = I32
        L.quest_test_step_fault.argtypes = [I32, I32]
        L.quest_test_step_fault.restype = I32
        L.quest_get_device_error.argtypes = [P]
        L.quest_get_device_error.restype = I32
        L.quest_status_string.argtypes = [I32]
        L.quest_status_string.restype = ctypes.c_char_p
        for fn in ("quest_append_kv", "quest_score_pages", "quest_select_topk",
                   "quest_sparse_decode_attn"):
            getattr(L, fn).restype = I32
        _lib = L
    return _lib


EXPORTED = ("quest_append_kv", "quest_score_pages", "quest_score_pages_per_head",
            "quest_select_topk", "quest_union_decode_attn", "quest_union_workspace_size",
            "quest_sparse_decode_attn", "quest_sparse_decode_attn_noalloc",
            "quest_attn_workspace_size",
            "quest_decode_step", "quest_decode_workspace_size", "quest_decode_step_kernel",
            "quest_recall_diagnostics", "quest_diag_workspace_size",
            "quest_rope_append_kv", "quest_dense_decode_attn",
            "quest_dense_decode_workspace_size", "quest_prefill_attn",
            "quest_prefill_workspace_size", "quest_norm_rope_append_kv",
            "quest_quant_page_bytes", "quest_quant_append_kv", "quest_quant_read_kv",
            "quest_quant_sparse_decode_attn", "quest_quant_dense_decode_attn",
            "quest_quant_decode_workspace_size", "quest_set_trace",
            "quest_test_step_fault", "quest_get_device_error", "quest_status_string")


def _check(status: int) -> None:
    if status != 0:
        raise RuntimeError(lib().quest_status_string(status).decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float16:
        return QUEST_F16
    if dt == torch.float32:
        return QUEST_F32
    raise ValueError(f"unsupported element type {dt}")


def _common_device(*tensors) -> int:
    """The CUDA device index that all have, else -1."""
    dev = tensors[0].get_device()
    return dev if all(t.get_device() == dev for t in tensors) else -1


class PagedCache:
    """One layer's pool + summary (caller-owned torch tensors).

    k_pool, v_pool: [n_phys, h_kv, page_size, head_dim]; summary:
    [n_phys, h_kv, 2, head_dim] (index 0 = min, 1 = max), either in the K/V
    dtype or, as a torch.uint8 tensor, E4M3 codes with directed rounding
    (fp16 K/V only; see summary_fp8 in quest.h).
    """

    def __init__(self, k_pool, v_pool, summary):
        self.k_pool, self.v_pool, self.summary = k_pool, v_pool, summary
        n_phys, h_kv, S, d = k_pool.shape
        self.n_phys, self.h_kv, self.page_size, self.head_dim = n_phys, h_kv, S, d
        self.dtype = k_pool.dtype
        self.device_index = _common_device(k_pool, v_pool, summary)
        self.summary_fp8 = summary.dtype == torch.uint8
        if not self.summary_fp8 and summary.dtype != k_pool.dtype:
            raise ValueError("summary must have the K/V dtype or be uint8 E4M3 codes")
        self.c = QuestCache(k_pool.data_ptr(), v_pool.data_ptr(), summary.data_ptr(),
                            n_phys, h_kv, S, d, dtype_code(k_pool.dtype), int(self.summary_fp8))

    @classmethod
    def empty(cls, n_phys, h_kv, page_size, head_dim, dtype, device="cuda", summary_fp8=False):
        kp = torch.empty((n_phys, h_kv, page_size, head_dim), dtype=dtype, device=device)
        vp = torch.empty_like(kp)
        sm = torch.empty((n_phys, h_kv, 2, head_dim), dtype=torch.uint8 if summary_fp8 else dtype,
                         device=device)
        return cls(kp, vp, sm)


class QuantCache:
    """One layer's pool of E4M3 records + summary (caller-owned torch tensors).

    pool: uint8 [n_phys, h_kv, quant_page_bytes(page_size, head_dim)] (the
    layout is quest_quant_cache's in quest.h; ``k_codes``, ``v_codes``,
    ``k_scales`` and ``v_scales`` are views of its parts, and its only exponents
    are -14 to 7); summary:
    [n_phys, h_kv, 2, head_dim], fp16 or, as torch.uint8, E4M3 codes. It goes
    to the quant_* calls and, for its summary, to the page scores; the calls
    that read fp16 or fp32 pages take the PagedCache of quant_read_kv.
    """

    dtype = torch.float16

    def __init__(self, pool, summary, page_size: int, head_dim: int):
        self.pool, self.summary = pool, summary
        n_phys, h_kv, _ = pool.shape
        self.n_phys, self.h_kv, self.page_size, self.head_dim = n_phys, h_kv, page_size, head_dim
        self.device_index = _common_device(pool, summary)
        self.summary_fp8 = summary.dtype == torch.uint8
        _expect("pool", pool, torch.uint8, (n_phys, h_kv, quant_page_bytes(page_size, head_dim)),
                pool.get_device())
        _expect("summary", summary, torch.uint8 if self.summary_fp8 else torch.float16,
                (n_phys, h_kv, 2, head_dim), pool.get_device())
        self.quant = QuestQuantCache(pool.data_ptr(), summary.data_ptr(), n_phys, h_kv, page_size,
                                     head_dim, int(self.summary_fp8))
        # what scoring takes: it reads the summary alone
        self.scored = QuestCache(pool.data_ptr(), pool.data_ptr(), summary.data_ptr(), n_phys, h_kv,
                                 page_size, head_dim, QUEST_F16, int(self.summary_fp8))

    @classmethod
    def empty(cls, n_phys, h_kv, page_size, head_dim, device="cuda", summary_fp8=False):
        pool = torch.empty((n_phys, h_kv, quant_page_bytes(page_size, head_dim)), dtype=torch.uint8,
                           device=device)
        summary = torch.empty((n_phys, h_kv, 2, head_dim), device=device,
                              dtype=torch.uint8 if summary_fp8 else torch.float16)
        return cls(pool, summary, page_size, head_dim)

    @property
    def c(self):
        raise TypeError("this call reads fp16 or fp32 pages: take the quant_* call, or a PagedCache "
                        "filled by quant_read_kv")

    def _part(self, start, size, dtype):
        return self.pool[..., start:start + size].view(dtype)

    @property
    def k_codes(self):
        """[n_phys, h_kv, head_dim / 64, page_size, 64], torch.float8_e4m3fn."""
        n = self.page_size * self.head_dim
        return self._part(0, n, torch.float8_e4m3fn).unflatten(-1, (self.head_dim // 64, self.page_size, 64))

    @property
    def v_codes(self):
        """[n_phys, h_kv, page_size / 16, head_dim / 32, 8, 4, 4, 2, 2], torch.float8_e4m3fn:
        dim 32 i + 4 g + c of token 16 s + 8 hi + 2 t + lo at [s, i, g, t, c, hi, lo]."""
        n = self.page_size * self.head_dim
        return self._part(n, n, torch.float8_e4m3fn).unflatten(
            -1, (self.page_size // 16, self.head_dim // 32, 8, 4, 4, 2, 2))

    @property
    def k_scales(self):
        """[n_phys, h_kv, page_size], torch.float8_e8m0fnu."""
        return self._part(2 * self.page_size * self.head_dim, self.page_size, torch.float8_e8m0fnu)

    @property
    def v_scales(self):
        """[n_phys, h_kv, page_size], torch.float8_e8m0fnu."""
        return self._part((2 * self.head_dim + 1) * self.page_size, self.page_size, torch.float8_e8m0fnu)


class PageTable:
    """Ragged page table on the device: page_indptr [B+1], page_indices [nnz],
    seq_lens [B] (int32). ``nnz`` is kept on the host."""

    def __init__(self, page_indptr, page_indices, seq_lens, nnz=None):
        self.page_indptr, self.page_indices, self.seq_lens = page_indptr, page_indices, seq_lens
        self.device_index = _common_device(page_indptr, page_indices, seq_lens)
        self.batch = int(seq_lens.shape[0])
        self.nnz = int(page_indices.shape[0]) if nnz is None else int(nnz)
        self.c = QuestPages(page_indptr.data_ptr(), page_indices.data_ptr(),
                            seq_lens.data_ptr(), self.batch, self.nnz)


def append_kv(cache: PagedCache, table: PageTable, k_new, v_new, append_indptr,
              seq_lens_before, stream=None) -> None:
    """quest_append_kv: write k_new/v_new [n_new, h_kv, d] into the pool and
    update the page min/max summaries."""
    _check(lib().quest_append_kv(ctypes.byref(cache.c), ctypes.byref(table.c),
                                 _ptr(k_new), _ptr(v_new), int(k_new.shape[0]),
                                 _ptr(append_indptr), _ptr(seq_lens_before),
                                 _stream(stream)))


def _scored(cache) -> QuestCache:
    return cache.scored if isinstance(cache, QuantCache) else cache.c


def score_pages(cache: PagedCache | QuantCache, table: PageTable, q, group: int, scores=None,
                stream=None):
    """quest_score_pages: scores [h_kv, nnz] fp32 of every page-table entry."""
    if scores is None:
        scores = torch.empty((cache.h_kv, table.nnz), dtype=torch.float32, device=q.device)
    _check(lib().quest_score_pages(ctypes.byref(_scored(cache)), ctypes.byref(table.c), _ptr(q),
                                   int(group), _ptr(scores), _stream(stream)))
    return scores


def score_pages_per_head(cache: PagedCache | QuantCache, table: PageTable, q, group: int, scores=None,
                         stream=None):
    """quest_score_pages_per_head: scores [h_kv * group, nnz] fp32, one row per
    query head (no group max)."""
    if scores is None:
        scores = torch.empty((cache.h_kv * group, table.nnz), dtype=torch.float32, device=q.device)
    _check(lib().quest_score_pages_per_head(ctypes.byref(_scored(cache)), ctypes.byref(table.c), _ptr(q),
                                            int(group), _ptr(scores), _stream(stream)))
    return scores


def union_workspace_size(batch, h_kv, group, head_dim, page_size, dtype, k) -> int:
    return int(lib().quest_union_workspace_size(batch, h_kv, group, head_dim, page_size,
                                                dtype_code(dtype), k))


def union_decode_attn(cache: PagedCache, table: PageTable, q, group: int, sel_logical, k: int,
                      out=None, lse=None, sm_scale: float = 0.0, union=None, workspace=None,
                      stream=None):
    """quest_union_decode_attn: per-query-head page sets sel_logical
    [B, h_q, k]; returns (out [B, h_q, d], lse [B, h_q], (union_logical
    [B, h_kv, group * k], union_mask uint8 [B, h_kv, group * k], union_count
    [B, h_kv]))."""
    B, h_q, d = q.shape
    dev = q.device
    h_kv = cache.h_kv
    if out is None:
        out = torch.empty((B, h_q, d), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((B, h_q), dtype=torch.float32, device=dev)
    if union is None:
        union = (torch.empty((B, h_kv, group * k), dtype=torch.int32, device=dev),
                 torch.empty((B, h_kv, group * k), dtype=torch.uint8, device=dev),
                 torch.empty((B, h_kv), dtype=torch.int32, device=dev))
    if workspace is None:
        n = union_workspace_size(B, h_kv, group, d, cache.page_size, cache.dtype, k)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    ul, um, uc = union
    _check(lib().quest_union_decode_attn(
        ctypes.byref(cache.c), ctypes.byref(table.c), _ptr(q), int(group), _ptr(sel_logical),
        int(k), _ptr(out), _ptr(lse), float(sm_scale), _ptr(ul), _ptr(um), _ptr(uc),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()), _stream(stream)))
    return out, lse, union


def select_topk(table: PageTable, h_kv: int, page_size: int, scores, k: int,
                out=None, stream=None, n_sink: int = 0, n_local: int = 0):
    """quest_select_topk: (sel_logical, sel_phys [B, h_kv, k], sel_count [B, h_kv]).
    n_sink / n_local: first / last valid pages always kept (hybrid budget)."""
    if out is None:
        dev = scores.device
        out = (torch.empty((table.batch, h_kv, k), dtype=torch.int32, device=dev),
               torch.empty((table.batch, h_kv, k), dtype=torch.int32, device=dev),
               torch.empty((table.batch, h_kv), dtype=torch.int32, device=dev))
    sl, sp, sc = out
    _check(lib().quest_select_topk(ctypes.byref(table.c), int(h_kv), int(page_size),
                                   _ptr(scores), int(k), int(n_sink), int(n_local),
                                   _ptr(sl), _ptr(sp), _ptr(sc), _stream(stream)))
    return sl, sp, sc


def attn_workspace_size(batch, h_kv, group, head_dim, page_size, k) -> int:
    return int(lib().quest_attn_workspace_size(batch, h_kv, group, head_dim, page_size, k))


def sparse_decode_attn(cache: PagedCache, table: PageTable, q, group: int, sel_logical,
                       sel_phys, k: int, out=None, lse=None, sm_scale: float = 0.0,
                       workspace=None, stream=None):
    """quest_sparse_decode_attn: (out [B, h_q, d] fp32, lse [B, h_q] fp32)."""
    B, h_q, d = q.shape
    dev = q.device
    if out is None:
        out = torch.empty((B, h_q, d), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((B, h_q), dtype=torch.float32, device=dev)
    if workspace is None:
        n = attn_workspace_size(B, cache.h_kv, group, d, cache.page_size, k)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    _check(lib().quest_sparse_decode_attn(
        ctypes.byref(cache.c), ctypes.byref(table.c), _ptr(q), int(group), _ptr(sel_logical),
        _ptr(sel_phys), int(k), _ptr(out), _ptr(lse), float(sm_scale), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream)))
    return out, lse


def diag_workspace_size(h_kv, group, nnz, page_size) -> int:
    return int(lib().quest_diag_workspace_size(h_kv, group, nnz, page_size))


def recall_diagnostics(cache: PagedCache, table: PageTable, q, group: int, sel_logical,
                       k: int, top_r: int, sm_scale: float = 0.0, workspace=None, stream=None):
    """quest_recall_diagnostics: dict of slack [h_q, nnz], eps [B, h_q],
    topr [B, h_q] and vmax [B, h_kv] (fp32)."""
    B, h_q, d = q.shape
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(slack=torch.empty((h_q, table.nnz), **f32), eps=torch.empty((B, h_q), **f32),
               topr=torch.empty((B, h_q), **f32), vmax=torch.empty((B, cache.h_kv), **f32))
    if workspace is None:
        n = diag_workspace_size(cache.h_kv, group, table.nnz, cache.page_size)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    _check(lib().quest_recall_diagnostics(
        ctypes.byref(cache.c), ctypes.byref(table.c), _ptr(q), int(group), _ptr(sel_logical),
        int(k), int(top_r), float(sm_scale), _ptr(out["slack"]), _ptr(out["eps"]),
        _ptr(out["topr"]), _ptr(out["vmax"]), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream)))
    return out


def decode_workspace_size(batch, nnz, h_kv, group, head_dim, page_size, dtype, k) -> int:
    return int(lib().quest_decode_workspace_size(batch, nnz, h_kv, group, head_dim, page_size,
                                                 dtype_code(dtype), k))


class DecodeStep:
    """Buffers of quest_decode_step for a fixed problem shape: scores,
    selections, outputs and a zero-filled workspace (reused across calls).
    n_sink / n_local: first / last valid pages always kept (hybrid budget)."""

    def __init__(self, cache: PagedCache, table: PageTable, group: int, k: int, device=None,
                 n_sink: int = 0, n_local: int = 0):
        cache.c                                                 # a QuantCache says here what it is not
        dev = device or cache.k_pool.device
        B, h = table.batch, cache.h_kv
        self.group, self.k = group, k
        self.n_sink, self.n_local = n_sink, n_local
        self.scores = torch.empty((h, max(table.nnz, 1)), dtype=torch.float32, device=dev)
        self.sel = (torch.empty((B, h, k), dtype=torch.int32, device=dev),
                    torch.empty((B, h, k), dtype=torch.int32, device=dev),
                    torch.empty((B, h), dtype=torch.int32, device=dev))
        self.out = torch.empty((B, h * group, cache.head_dim), dtype=torch.float32, device=dev)
        self.lse = torch.empty((B, h * group), dtype=torch.float32, device=dev)
        n = decode_workspace_size(B, table.nnz, h, group, cache.head_dim, cache.page_size,
                                  cache.dtype, k)
        if n == 0:
            raise RuntimeError("quest_decode_step does not support this shape")
        self.workspace = torch.zeros(n, dtype=torch.uint8, device=dev)

    def __call__(self, cache: PagedCache, table: PageTable, q, k_new=None, v_new=None,
                 sm_scale: float = 0.0, stream=None):
        sl, sp, sc = self.sel
        _check(lib().quest_decode_step(
            ctypes.byref(cache.c), ctypes.byref(table.c), _ptr(k_new), _ptr(v_new), _ptr(q),
            int(self.group), int(self.k), int(self.n_sink), int(self.n_local),
            _ptr(self.scores), _ptr(sl), _ptr(sp), _ptr(sc),
            _ptr(self.out), _ptr(self.lse), float(sm_scale), _ptr(self.workspace),
            int(self.workspace.numel()), _stream(stream)))
        return self.out, self.lse


def decode_step_kernel(batch, h_kv, group, head_dim, page_size, dtype, k, summary_fp8=False) -> str:
    """quest_decode_step_kernel: the kernel quest_decode_step launches for
    these sizes on the current device ("cstep_kernel", "step_kernel", or ""
    if unsupported)."""
    r = int(lib().quest_decode_step_kernel(int(batch), int(h_kv), int(group), int(head_dim),
                                           int(page_size), dtype_code(dtype), int(k),
                                           int(bool(summary_fp8))))
    return {2: "cstep_kernel", 1: "step_kernel"}.get(r, "")


def rope_frequencies(rotary_dim: int, base: float = 10000.0, device="cuda"):
    """Angles per position of the plain rotation, base^(-2j / rotary_dim): fp64
    [rotary_dim / 2]. Scaled variants are any other fp64 tensor of that shape."""
    j = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device)
    return base ** (-j / rotary_dim)


def _expect(name, t, dtype, shape, device):
    """Raises unless t is a contiguous tensor of this type, shape and CUDA device index."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {tuple(shape)} on CUDA device {device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device} with strides {t.stride()}")


def _expect_rows(name, t, dtype, shape, device) -> int:
    """Raises unless t [n, heads, d] has this type, shape and CUDA device index and
    dense rows, maybe apart; returns the elements from one row to the next."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device:
        n, row, d = shape[0], shape[1] * shape[2], shape[2]
        s0, s1, s2 = t.stride()
        if n == 0 or (n == 1 or s0 >= row) and s2 == 1 and (s1 == d or shape[1] == 1):
            return s0 if n > 1 else row
    raise ValueError(f"{name} must be {dtype} {tuple(shape)} on CUDA device {device} with contiguous "
                     f"rows, not {t.dtype} {tuple(t.shape)} on {t.device} with strides {t.stride()}")


def _current(cache: PagedCache | QuantCache, table: PageTable) -> int:
    """Index of the current device, which has to hold the cache and its page table."""
    dev = cache.device_index
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"the cache must be on the current CUDA device, not {cache.summary.device}")
    if table.device_index != dev:
        raise ValueError(f"the page table must be on CUDA device {dev}, not {table.seq_lens.device}")
    return dev


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream must be of CUDA device {dev}, not {stream.device_index}")
    return stream.cuda_stream


def _result(shape, dtype, dev, stream):
    """Memory for a result that ``stream`` writes: taken from that stream, so no
    earlier work of the current one still uses it, and kept, when it is
    released, until the current stream has read it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _expect_workspace(t, device):
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"the workspace must be contiguous on CUDA device {device}, not on {t.device} "
                         f"with strides {t.stride()}")


def _scratch(n, dev, stream):
    """A workspace from the memory of the stream that will use it."""
    with torch.cuda.stream(stream):
        return torch.empty(max(n, 16), dtype=torch.uint8, device=dev)


def rope_append_kv(cache: PagedCache, table: PageTable, q, k_new, v_new, append_indptr,
                   seq_lens_before, inv_freq, group: int, q_out=None, positions=None,
                   interleaved: bool = False, stream=None):
    """quest_rope_append_kv: rotates k_new [n_new, h_kv, d] into the pages with
    v_new, updates the summaries, and returns q [n_new, h_kv * group, d]
    rotated (q may be None). Tokens may be strided (the parts of one fused
    projection); inv_freq is fp64 [rotary_dim / 2] (see rope_frequencies);
    positions int32 [n_new] replaces the tokens' places in the cache. In a loop
    of small calls pass q_out: its allocation is 6 of their 15 us on the host."""
    dev, dt, n = _current(cache, table), cache.dtype, k_new.shape[0]
    h, d = cache.h_kv, cache.head_dim
    kv = (n, h, d)
    k_stride = _expect_rows("k_new", k_new, dt, kv, dev)
    v_stride = _expect_rows("v_new", v_new, dt, kv, dev)
    _expect("append_indptr", append_indptr, torch.int32, (table.batch + 1,), dev)
    _expect("seq_lens_before", seq_lens_before, torch.int32, (table.batch,), dev)
    _expect("inv_freq", inv_freq, torch.float64, (inv_freq.numel(),), dev)
    if positions is not None:
        _expect("positions", positions, torch.int32, (n,), dev)
    q_stride = 0
    if q is not None:
        rows = (n, h * group, d)
        q_stride = _expect_rows("q", q, dt, rows, dev)
        if q_out is None:
            q_out = _result(rows, dt, dev, stream)
        _expect("q_out", q_out, dt, rows, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    rope = QuestRope(_ptr(inv_freq), _ptr(positions), 2 * inv_freq.numel(), int(bool(interleaved)))
    _check(lib().quest_rope_append_kv(
        ctypes.byref(cache.c), ctypes.byref(table.c), ctypes.byref(rope), _ptr(q), _ptr(k_new),
        _ptr(v_new), q_stride, k_stride, v_stride, n, int(group), _ptr(append_indptr),
        _ptr(seq_lens_before), _ptr(q_out), _raw_stream(stream, dev)))
    return q_out


class QKNorm:
    """quest_qk_norm: device fp32 weights [d], or [heads, d] for one per head
    (either may be None: that side is not normed), kept alive here."""

    def __init__(self, q_weight, k_weight, eps: float = 1e-6):
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, float(eps)
        self.sides = []                 # (name, heads or 0 for all, dims, device) of each weight
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                if w.dim() not in (1, 2):
                    raise ValueError(f"{name} must be [d] or [heads, d], not {tuple(w.shape)}")
                _expect(name, w, torch.float32, tuple(w.shape), w.get_device())
                self.sides.append((name, w.shape[0] if w.dim() == 2 else 0, w.shape[-1], w.get_device()))
        per_head = [int(w is not None and w.dim() == 2) for w in (q_weight, k_weight)]
        self.c = QuestQKNorm(_ptr(q_weight), _ptr(k_weight), *per_head, self.eps)

    def check(self, h_q, h_kv, d, device):
        for name, heads, dims, dev in self.sides:
            if dims != d or dev != device or heads and heads != (h_q if name == "q_weight" else h_kv):
                raise ValueError(f"{name} must have {d} dims for {h_q} query and {h_kv} KV heads on CUDA device "
                                 f"{device}, not {dims} for {heads or 'all'} heads on {dev}")


def _append_args(cache, table, q, k_new, v_new, append_indptr, seq_lens_before, inv_freq, group,
                 q_out, positions, interleaved, stream, dev):
    """Checks what the normed and the E4M3 append share: (QuestRope or None,
    q_out, the arguments of the C calls from q on). In a decode loop the calls
    are bound by these checks on the host, so what is as usual is looked at in
    one place, and the helpers only where something is not."""
    dt, h, d, i32 = cache.dtype, cache.h_kv, cache.head_dim, torch.int32
    kv = k_new.shape
    n = kv[0]
    (ks, k1, k2), (vs, v1, v2) = k_new.stride(), v_new.stride()
    if not (n > 1 and kv == (n, h, d) and v_new.shape == kv and k_new.dtype is dt and v_new.dtype is dt and
            k_new.get_device() == dev and v_new.get_device() == dev and
            k2 == v2 == 1 and k1 == v1 == d and ks >= h * d and vs >= h * d):
        ks = _expect_rows("k_new", k_new, dt, (n, h, d), dev)
        vs = _expect_rows("v_new", v_new, dt, (n, h, d), dev)
    B = table.batch
    if not (append_indptr.dtype is i32 and append_indptr.shape == (B + 1,) and append_indptr.get_device() == dev and
            append_indptr.is_contiguous() and seq_lens_before.dtype is i32 and seq_lens_before.shape == (B,) and
            seq_lens_before.get_device() == dev and seq_lens_before.is_contiguous()):
        _expect("append_indptr", append_indptr, i32, (B + 1,), dev)
        _expect("seq_lens_before", seq_lens_before, i32, (B,), dev)
    rope = None
    if inv_freq is not None:
        half = inv_freq.numel()
        _expect("inv_freq", inv_freq, torch.float64, (half,), dev)
        if positions is not None:
            _expect("positions", positions, i32, (n,), dev)
        rope = QuestRope(inv_freq.data_ptr(), _ptr(positions), 2 * half, 1 if interleaved else 0)
    elif positions is not None:
        raise ValueError("positions need inv_freq")
    q_stride = 0
    if q is not None:
        rows = (n, h * group, d)
        q_stride = _expect_rows("q", q, dt, rows, dev)
        if q_out is None:
            q_out = _result(rows, dt, dev, stream)
        _expect("q_out", q_out, dt, rows, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    return rope, q_out, (_ptr(q), k_new.data_ptr(), v_new.data_ptr(), q_stride, ks, vs, n, group,
                         append_indptr.data_ptr(), seq_lens_before.data_ptr(), _ptr(q_out), _raw_stream(stream, dev))


def norm_rope_append_kv(cache: PagedCache, table: PageTable, q, k_new, v_new, append_indptr,
                        seq_lens_before, norm: QKNorm, group: int, inv_freq=None, q_out=None,
                        positions=None, interleaved: bool = False, stream=None):
    """quest_norm_rope_append_kv: rope_append_kv with every query and key head
    normed before the rotation, in the same pass; inv_freq None: no rotation.
    Returns the queries (or None)."""
    dev = _current(cache, table)
    norm.check(cache.h_kv * group, cache.h_kv, cache.head_dim, dev)
    rope, q_out, tail = _append_args(cache, table, q, k_new, v_new, append_indptr, seq_lens_before,
                                     inv_freq, group, q_out, positions, interleaved, stream, dev)
    _check(lib().quest_norm_rope_append_kv(
        ctypes.byref(cache.c), ctypes.byref(table.c), None if rope is None else ctypes.byref(rope),
        ctypes.byref(norm.c), *tail))
    return q_out


def quant_page_bytes(page_size: int, head_dim: int) -> int:
    """Bytes of one page of one KV head in a QuantCache (0: unsupported sizes)."""
    return int(lib().quest_quant_page_bytes(page_size, head_dim))


def quant_append_kv(cache: QuantCache, table: PageTable, q, k_new, v_new, append_indptr,
                    seq_lens_before, group: int, inv_freq=None, norm: QKNorm | None = None,
                    q_out=None, positions=None, interleaved: bool = False, stream=None):
    """quest_quant_append_kv: k_new and v_new [n_new, h_kv, d] (fp16) into the
    records and the page summaries; keys and queries normed (norm) and rotated
    (inv_freq) on the way, as in norm_rope_append_kv. With neither, q has to be
    None. Returns the queries (or None)."""
    dev = _current(cache, table)
    if norm is not None:
        norm.check(cache.h_kv * group, cache.h_kv, cache.head_dim, dev)
    rope, q_out, tail = _append_args(cache, table, q, k_new, v_new, append_indptr, seq_lens_before,
                                     inv_freq, group, q_out, positions, interleaved, stream, dev)
    _check(lib().quest_quant_append_kv(
        ctypes.byref(cache.quant), ctypes.byref(table.c), None if rope is None else ctypes.byref(rope),
        None if norm is None else ctypes.byref(norm.c), *tail))
    return q_out


def quant_read_kv(cache: QuantCache, table: PageTable, dst: PagedCache, dst_indices=None,
                  stream=None) -> None:
    """quest_quant_read_kv: the numbers that the cache holds into dst's pages:
    table entry e to page dst_indices[e] (int32 [nnz]; None: page e). dst's
    summary is left as it is."""
    dev = _current(cache, table)
    if (dst.dtype is not torch.float16 or dst.device_index != dev or
            (dst.h_kv, dst.page_size, dst.head_dim) != (cache.h_kv, cache.page_size, cache.head_dim)):
        raise ValueError(f"dst must be a fp16 PagedCache of {cache.h_kv} heads, pages of {cache.page_size} "
                         f"and {cache.head_dim} dims on CUDA device {dev}")
    if dst_indices is not None:
        _expect("dst_indices", dst_indices, torch.int32, (table.nnz,), dev)
    _check(lib().quest_quant_read_kv(
        ctypes.byref(cache.quant), ctypes.byref(table.c), _ptr(dst.k_pool), _ptr(dst.v_pool), dst.n_phys,
        _ptr(dst_indices), _raw_stream(stream, dev)))


def quant_decode_workspace_size(batch, h_kv, group, head_dim, page_size) -> int:
    return int(lib().quest_quant_decode_workspace_size(batch, h_kv, group, head_dim, page_size))


def _quant_decode_args(cache, table, q, group, out, lse, workspace, stream, dev):
    """(out, lse, workspace) of a decode call, checked (as in _append_args)."""
    f32 = torch.float32
    B, h_q, d = table.batch, cache.h_kv * group, cache.head_dim
    rows, heads = (B, h_q, d), (B, h_q)
    if out is None:
        out = _result(rows, f32, dev, stream)
    if lse is None:
        lse = _result(heads, f32, dev, stream)
    if not (q.dtype is torch.float16 and out.dtype is f32 and lse.dtype is f32 and q.shape == rows and
            out.shape == rows and lse.shape == heads and q.is_contiguous() and out.is_contiguous() and
            lse.is_contiguous() and q.get_device() == dev and out.get_device() == dev and lse.get_device() == dev):
        _expect("q", q, torch.float16, rows, dev)
        _expect("out", out, f32, rows, dev)
        _expect("lse", lse, f32, heads, dev)
    if workspace is None:
        workspace = _scratch(quant_decode_workspace_size(B, cache.h_kv, group, d, cache.page_size), dev, stream)
    _expect_workspace(workspace, dev)
    return out, lse, workspace


def quant_sparse_decode_attn(cache: QuantCache, table: PageTable, q, group: int, sel_logical, sel_phys,
                             k: int, out=None, lse=None, sm_scale: float = 0.0, workspace=None,
                             stream=None):
    """quest_quant_sparse_decode_attn: (out [B, h_q, d] fp32, lse [B, h_q] fp32)
    over the pages that select_topk chose (int32 [B, h_kv, k]). ``workspace``:
    uint8, quant_decode_workspace_size bytes."""
    dev = _current(cache, table)
    lists, i32 = (table.batch, cache.h_kv, k), torch.int32
    if not (sel_logical.dtype is i32 and sel_phys.dtype is i32 and sel_logical.shape == lists and
            sel_phys.shape == lists and sel_logical.is_contiguous() and sel_phys.is_contiguous() and
            sel_logical.get_device() == dev and sel_phys.get_device() == dev):
        _expect("sel_logical", sel_logical, i32, lists, dev)
        _expect("sel_phys", sel_phys, i32, lists, dev)
    out, lse, workspace = _quant_decode_args(cache, table, q, group, out, lse, workspace, stream, dev)
    _check(lib().quest_quant_sparse_decode_attn(
        ctypes.byref(cache.quant), ctypes.byref(table.c), q.data_ptr(), group, sel_logical.data_ptr(),
        sel_phys.data_ptr(), k, out.data_ptr(), lse.data_ptr(), sm_scale, workspace.data_ptr(), workspace.nbytes,
        _raw_stream(stream, dev)))
    return out, lse


def quant_dense_decode_attn(cache: QuantCache, table: PageTable, q, group: int, out=None, lse=None,
                            sm_scale: float = 0.0, mods: ScoreMods | None = None, workspace=None,
                            stream=None):
    """quest_quant_dense_decode_attn: (out [B, h_q, d] fp32, lse [B, h_q] fp32)
    of one query per request over all of its cached tokens. ``workspace``: as
    quant_sparse_decode_attn."""
    dev = _current(cache, table)
    if mods is not None:
        mods.check(cache.h_kv * group, table.batch, table.batch, dev)
    out, lse, workspace = _quant_decode_args(cache, table, q, group, out, lse, workspace, stream, dev)
    _check(lib().quest_quant_dense_decode_attn(
        ctypes.byref(cache.quant), ctypes.byref(table.c), q.data_ptr(), group,
        None if mods is None else ctypes.byref(mods.c), out.data_ptr(), lse.data_ptr(), sm_scale,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, dev)))
    return out, lse


class ScoreMods:
    """quest_score_mods: softcap, window, and device tensors alibi_slopes fp32
    [h_q], doc_starts int32 [query rows], prefix_lens int32 [batch] (each may be
    None), kept alive here."""

    def __init__(self, softcap: float = 0.0, window: int = 0, alibi_slopes=None, doc_starts=None,
                 prefix_lens=None):
        self.softcap, self.window = float(softcap), int(window)
        if abs(self.window) >= 1 << 31:
            raise ValueError("window must fit 32 bits")
        self.alibi_slopes, self.doc_starts, self.prefix_lens = alibi_slopes, doc_starts, prefix_lens
        self.c = QuestScoreMods(_ptr(alibi_slopes), _ptr(doc_starts), _ptr(prefix_lens),
                                self.softcap, self.window)

    def check(self, h_q, rows, batch, device):
        if self.alibi_slopes is not None:
            _expect("alibi_slopes", self.alibi_slopes, torch.float32, (h_q,), device)
        if self.doc_starts is not None:
            _expect("doc_starts", self.doc_starts, torch.int32, (rows,), device)
        if self.prefix_lens is not None:
            _expect("prefix_lens", self.prefix_lens, torch.int32, (batch,), device)


def dense_decode_workspace_size(batch, nnz, h_kv, group, head_dim, page_size, dtype) -> int:
    return int(lib().quest_dense_decode_workspace_size(batch, nnz, h_kv, group, head_dim,
                                                       page_size, dtype_code(dtype)))


def dense_decode_attn(cache: PagedCache, table: PageTable, q, group: int, out=None, lse=None,
                      sm_scale: float = 0.0, mods: ScoreMods | None = None, workspace=None,
                      stream=None):
    """quest_dense_decode_attn: (out [B, h_q, d] fp32, lse [B, h_q] fp32) of one
    query per request over all of its cached tokens. ``workspace``: uint8,
    dense_decode_workspace_size bytes."""
    dev, h_q, d = _current(cache, table), cache.h_kv * group, cache.head_dim
    B = table.batch
    _expect("q", q, cache.dtype, (B, h_q, d), dev)
    if out is None:
        out = _result((B, h_q, d), torch.float32, dev, stream)
    if lse is None:
        lse = _result((B, h_q), torch.float32, dev, stream)
    _expect("out", out, torch.float32, (B, h_q, d), dev)
    _expect("lse", lse, torch.float32, (B, h_q), dev)
    if mods is not None:
        mods.check(h_q, B, B, dev)
    if workspace is None:
        n = dense_decode_workspace_size(B, table.nnz, cache.h_kv, group, d, cache.page_size,
                                        cache.dtype)
        workspace = _scratch(n, dev, stream)
    _expect_workspace(workspace, dev)
    _check(lib().quest_dense_decode_attn(
        ctypes.byref(cache.c), ctypes.byref(table.c), _ptr(q), int(group),
        None if mods is None else ctypes.byref(mods.c), _ptr(out), _ptr(lse), float(sm_scale),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()), _raw_stream(stream, dev)))
    return out, lse


def prefill_workspace_size(batch, n_q, nnz, h_kv, group, head_dim, page_size, dtype) -> int:
    return int(lib().quest_prefill_workspace_size(batch, n_q, nnz, h_kv, group, head_dim,
                                                  page_size, dtype_code(dtype)))


def prefill_attn(cache: PagedCache, table: PageTable, q, group: int, q_indptr, out=None, lse=None,
                 sm_scale: float = 0.0, mods: ScoreMods | None = None, workspace=None,
                 stream=None):
    """quest_prefill_attn: (out [n_q, h_q, d] in the cache's type, lse [n_q, h_q]
    fp32) of each request's last tokens, rows q_indptr[r] .. q_indptr[r + 1] of
    q, over its cached tokens. ``workspace``: uint8, prefill_workspace_size
    bytes."""
    dev, h_q, d = _current(cache, table), cache.h_kv * group, cache.head_dim
    n = q.shape[0]
    _expect("q", q, cache.dtype, (n, h_q, d), dev)
    _expect("q_indptr", q_indptr, torch.int32, (table.batch + 1,), dev)
    if out is None:
        out = _result((n, h_q, d), cache.dtype, dev, stream)
    if lse is None:
        lse = _result((n, h_q), torch.float32, dev, stream)
    _expect("out", out, cache.dtype, (n, h_q, d), dev)
    _expect("lse", lse, torch.float32, (n, h_q), dev)
    if mods is not None:
        mods.check(h_q, n, table.batch, dev)
    if workspace is None:
        size = prefill_workspace_size(table.batch, n, table.nnz, cache.h_kv, group, d,
                                      cache.page_size, cache.dtype)
        workspace = _scratch(size, dev, stream)
    _expect_workspace(workspace, dev)
    _check(lib().quest_prefill_attn(
        ctypes.byref(cache.c), ctypes.byref(table.c), _ptr(q), int(group), _ptr(q_indptr), int(n),
        None if mods is None else ctypes.byref(mods.c), _ptr(out), _ptr(lse), float(sm_scale),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()), _raw_stream(stream, dev)))
    return out, lse


TRACE_NAMES = ("start", "scored", "selected", "att_start", "att_pages", "att_merged",
               "sel_begin", "sel_end", "", "exit",
               "sel0_polled | desc0", "sel0_done | page0", "sel1_polled | merged",
               "sel1_done | fmerge0", "sel2_polled | fmerge1", "sel2_done")
# slots 6-7: the first select's start (after the scored gate) and the last
# select's end, on every CTA that selects; slots 10-15 depend on the CTA's
# role: select stamps on dedicated selectors (the CTAs whose "scored" stamp
# precedes any scoring), attention and final-merge stamps on the others

# the cluster kernel's slots (unused ones empty)
CTRACE_NAMES = ("start", "prev_waited", "", "", "att_tile0", "keys_in", "sel_published",
                "merged_last", "", "exit", "topk_done", "phys_done", "", "", "", "")


def set_trace(buffer, max_ctas=0, batch=0, h_kv=0, group=1, head_dim=128, page_size=16,
              dtype=torch.float16, k=1) -> int:
    """quest_set_trace: per-CTA phase stamps of later decode steps into
    `buffer` (uint64 device tensor of 16 * max_ctas entries); None disables.
    Returns the grid size used for the given shape."""
    return int(lib().quest_set_trace(_ptr(buffer), int(max_ctas), int(batch), int(h_kv),
                                     int(group), int(head_dim), int(page_size),
                                     dtype_code(dtype), int(k)))


def sparse_decode_attn_noalloc(cache: PagedCache, table: PageTable, q, group: int,
                               sel_logical, sel_phys, k: int, out=None, lse=None,
                               sm_scale: float = 0.0, stream=None):
    """quest_sparse_decode_attn_noalloc: the same attention with the split-K
    partials in the library's fixed 4 MiB buffer (for callers that cannot
    allocate device memory); calls on overlapping streams race on it."""
    B, h_q, d = q.shape
    if out is None:
        out = torch.empty((B, h_q, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, h_q), dtype=torch.float32, device=q.device)
    _check(lib().quest_sparse_decode_attn_noalloc(
        ctypes.byref(cache.c), ctypes.byref(table.c), _ptr(q), int(group), _ptr(sel_logical),
        _ptr(sel_phys), int(k), _ptr(out), _ptr(lse), float(sm_scale), _stream(stream)))
    return out, lse


def test_step_fault(mode: int, wait_limit: int = 0) -> None:
    """quest_test_step_fault: mode 1 makes a wait of later decode steps on the
    cluster kernel run out, mode 2 one of later attention calls; under
    `wait_limit` tries per wait (0 = default). Mode 0 restores normal
    operation."""
    _check(lib().quest_test_step_fault(int(mode), int(wait_limit)))


def device_error(stream=None) -> int:
    """Synchronise and return (then clear) the device error word."""
    v = int(lib().quest_get_device_error(_stream(stream)))
    if v < 0:
        raise RuntimeError("quest_get_device_error: CUDA call failed")
    return v
