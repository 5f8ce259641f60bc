"""Python binding of libdsa (include/dsa.h): argument marshalling only.

Every function here has the name of the C entry point it calls, takes torch
tensors (device memory owned by torch) and passes their pointers, sizes and
the current CUDA stream.  No step of the DSA path runs in Python: if the
shared library is missing, importing this module raises.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE, DSA_ERR_CUDA, DSA_ERR_TIMEOUT, DSA_ERR_INDEX = range(7)
DSA_F32, DSA_BF16, DSA_E4M3 = 0, 1, 2
(DSA_OP_FOLD, DSA_OP_INDEX_SCORES, DSA_OP_TOPK, DSA_OP_SPARSE_ATTN, DSA_OP_FORWARD, DSA_OP_FORWARD_HOST,
 DSA_OP_NORM_ROPE_BWD, DSA_OP_PAGED_SELECT, DSA_OP_PAGED_ATTN) = range(9)

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libdsa.so not built ({LIB_PATH}); run python -m sparse_attention_11_b200.build")
_lib = ctypes.CDLL(LIB_PATH)

_P, _I32, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class dsa_seqs(ctypes.Structure):
    _fields_ = [("batch", _I32), ("total_q", _I64), ("total_k", _I64), ("max_seqlen_q", _I64),
                ("max_seqlen_k", _I64), ("cu_seqlens_q", _P), ("cu_seqlens_k", _P)]


class dsa_indexer_args(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("q_idx", _P), ("q_idx_scale", _P), ("w_dtype", _I32), ("w_index", _P),
                ("k_idx", _P), ("k_idx_scale", _P), ("k_per_row", _P)]


class dsa_attn_args(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("heads", _I32), ("dk", _I32), ("dv", _I32), ("q", _P), ("q_stride_tok", _I64),
                ("q_stride_head", _I64), ("k", _P), ("k_stride", _I64), ("v", _P), ("v_stride", _I64),
                ("scale", _F), ("out", _P), ("out_stride_tok", _I64), ("out_stride_head", _I64), ("lse", _P)]


class dsa_row_args(ctypes.Structure):
    _fields_ = [("norm_dim", _I32), ("eps", _F), ("weight", _P), ("rope_begin", _I32), ("rope_dim", _I32),
                ("rope_interleaved", _I32), ("cos_sin", _P), ("rope_positions", _I64)]


class dsa_pages(ctypes.Structure):
    _fields_ = [("page_size", _I32), ("num_pages", _I64), ("table", _P), ("ld_table", _I64), ("kv_page_stride", _I64),
                ("v_page_stride", _I64), ("idx_page_stride", _I64), ("scale_page_stride", _I64)]


class dsa_append_args(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("dim", _I32), ("kv_new", _P), ("kv_new_stride", _I64), ("kv", _P), ("kv_stride", _I64),
                ("kv_row", ctypes.POINTER(dsa_row_args)), ("idx_dtype", _I32), ("idx_new", _P), ("idx_new_stride", _I64),
                ("idx", _P), ("idx_scale", _P), ("idx_row", ctypes.POINTER(dsa_row_args))]


_S, _IA, _AA = ctypes.POINTER(dsa_seqs), ctypes.POINTER(dsa_indexer_args), ctypes.POINTER(dsa_attn_args)
_RA, _PG, _AP = ctypes.POINTER(dsa_row_args), ctypes.POINTER(dsa_pages), ctypes.POINTER(dsa_append_args)
_lib.dsa_status_string.restype = ctypes.c_char_p
_lib.dsa_status_string.argtypes = [ctypes.c_int]
_lib.dsa_version.restype = ctypes.c_int
_lib.dsa_workspace_size.argtypes = [ctypes.c_int, _S, _I32, _IA, _AA, ctypes.POINTER(_SZ)]
_lib.dsa_fold.argtypes = [_S, _IA, _P, _P, _P, _SZ, _P]
_lib.dsa_index_scores.argtypes = [_S, _IA, _I64, _I64, _P, _I64, _P, _SZ, _P]
_lib.dsa_topk.argtypes = [_S, _P, _I64, _I64, _I64, _I32, _P, _I64, _P, _SZ, _P]
_lib.dsa_sparse_attn.argtypes = [_S, _AA, _P, _I64, _I32, _P, _SZ, _P]
_lib.dsa_attn_target.argtypes = [_S, _AA, _P, _I64, _I32, _P, _I64, _P, _SZ, _P]
_lib.dsa_indexer_kl.argtypes = [_S, _P, _I64, _P, _P, _I64, _P, _I64, _I32, _P, _I64, _P, _P, _I64, _P, _P, _I64, _P,
                                _SZ, _P]
_lib.dsa_sparse_attn_bwd.argtypes = [_S, _AA, _P, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I64,
                                     _P, _SZ, _P]
_lib.dsa_forward.argtypes = [_S, _IA, _AA, _I32, _P, _I64, _P, _SZ, _P]
_lib.dsa_forward_host.argtypes = [_S, _IA, _AA, _I32, _P, _I64, _P, _SZ, _P, _P, _P]
_lib.dsa_select.argtypes = [_S, _IA, _I32, _P, _I64, _P, _SZ, _P]
_lib.dsa_select_noalloc.argtypes = [_S, _IA, _I32, _P, _I64, _P]
_lib.dsa_norm_rope.argtypes = [_S, _RA, _I32, _I32, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _SZ, _P]
_lib.dsa_norm_rope_bwd.argtypes = [_S, _RA, _I32, _I32, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _SZ,
                                   _P]
_lib.dsa_cache_append.argtypes = [_S, _PG, _AP, _P, _SZ, _P]
_lib.dsa_paged_scores.argtypes = [_S, _PG, _I32, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _P]
_lib.dsa_paged_select.argtypes = [_S, _PG, _IA, _I32, _P, _I64, _P, _SZ, _P]
_lib.dsa_paged_attn.argtypes = [_S, _PG, _AA, _P, _I64, _I32, _P, _SZ, _P]
_lib.dsa_sync_status.argtypes = [_P, _P, ctypes.POINTER(_I64)]
_lib.dsa_selftest_wait_timeout.argtypes = [_P, _SZ, _I64, _P]
for _f in ("dsa_workspace_size", "dsa_fold", "dsa_index_scores", "dsa_topk", "dsa_sparse_attn", "dsa_sparse_attn_bwd",
           "dsa_attn_target", "dsa_indexer_kl",
           "dsa_forward",
           "dsa_forward_host",
           "dsa_select", "dsa_select_noalloc",
           "dsa_norm_rope", "dsa_norm_rope_bwd", "dsa_cache_append", "dsa_paged_scores", "dsa_paged_select",
           "dsa_paged_attn",
           "dsa_sync_status", "dsa_selftest_wait_timeout"):
    getattr(_lib, _f).restype = ctypes.c_int

EXPORTED = ("dsa_status_string", "dsa_version", "dsa_workspace_size", "dsa_fold", "dsa_index_scores", "dsa_topk",
            "dsa_sparse_attn", "dsa_sparse_attn_bwd", "dsa_attn_target", "dsa_indexer_kl", "dsa_forward",
            "dsa_forward_host", "dsa_select",
            "dsa_select_noalloc", "dsa_norm_rope", "dsa_norm_rope_bwd", "dsa_cache_append", "dsa_paged_scores",
            "dsa_paged_select", "dsa_paged_attn", "dsa_sync_status",
            "dsa_selftest_wait_timeout")


class DsaError(RuntimeError):
    def __init__(self, code, where, detail=None):
        msg = f"{where}: {_lib.dsa_status_string(code).decode()} (status {code})"
        if detail is not None:
            msg += f", detail {detail}"
        super().__init__(msg)
        self.code = code
        self.detail = detail


_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream)


def _check(code, where):
    if code != DSA_OK:
        raise DsaError(code, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    """The current stream's handle (without torch.cuda.current_stream's object,
    which costs 3 us a call)."""
    if not torch.cuda._initialized:
        torch.cuda._lazy_init()
    return _raw_stream(_device())


def status_string(code):
    return _lib.dsa_status_string(code).decode()


def version():
    return _lib.dsa_version()


class Seqs:
    """Packed batch description; keeps the device cu_seqlens tensors alive."""

    def __init__(self, cu_q, cu_k, device="cuda"):
        cq = torch.as_tensor(cu_q, dtype=torch.int64)
        ck = torch.as_tensor(cu_k, dtype=torch.int64)
        lq, lk = (cq[1:] - cq[:-1]), (ck[1:] - ck[:-1])
        self.cu_q = cq.to(device)
        self.cu_k = ck.to(device)
        self.c = dsa_seqs(len(cq) - 1, int(cq[-1]), int(ck[-1]), int(lq.max()) if len(lq) else 0,
                          int(lk.max()) if len(lk) else 0, self.cu_q.data_ptr(), self.cu_k.data_ptr())
        self._index = self.cu_q.get_device()

    @property
    def total_q(self):
        return self.c.total_q

    @property
    def total_k(self):
        return self.c.total_k

    @property
    def max_seqlen_k(self):
        return self.c.max_seqlen_k


def indexer_args(q_idx, q_idx_scale, w_index, k_idx, k_idx_scale, k_per_row=None):
    """Indexer operands: float32 tensors (fp32 path) or uint8 e4m3 codes +
    float32 scales with a bfloat16 W (FP8 path); k_per_row: optional int32
    device tensor [total_q] of per-query k (dynamic k)."""
    fp8 = q_idx.dtype == torch.uint8
    a = dsa_indexer_args(DSA_E4M3 if fp8 else DSA_F32, q_idx.data_ptr(),
                         q_idx_scale.data_ptr() if q_idx_scale is not None else None,
                         DSA_BF16 if w_index.dtype == torch.bfloat16 else DSA_F32, w_index.data_ptr(),
                         k_idx.data_ptr(), k_idx_scale.data_ptr() if k_idx_scale is not None else None,
                         k_per_row.data_ptr() if k_per_row is not None else None)
    a._keep = (q_idx, q_idx_scale, w_index, k_idx, k_idx_scale, k_per_row)
    return a


def attn_args(q, k, v, scale, out, lse=None):
    """q [T,H,dk]; k [Tk,>=dk] (row stride k.stride(0)); v [Tk,>=dv] (may be a
    view of k's first columns); out [T,H,dv]; lse [T,H] or None."""
    dt = DSA_BF16 if q.dtype == torch.bfloat16 else DSA_F32
    a = dsa_attn_args(dt, q.shape[1], q.shape[2], out.shape[2], q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(),
                      k.stride(0), v.data_ptr(), v.stride(0), float(scale), out.data_ptr(), out.stride(0),
                      out.stride(1), lse.data_ptr() if lse is not None else None)
    a._keep = (q, k, v, out, lse)
    return a


def dsa_workspace_size(op, seqs, k=0, ia=None, aa=None):
    n = _SZ(0)
    _check(_lib.dsa_workspace_size(op, ctypes.byref(seqs.c), k, ctypes.byref(ia) if ia is not None else None,
                                   ctypes.byref(aa) if aa is not None else None, ctypes.byref(n)), "dsa_workspace_size")
    return n.value


def workspace(nbytes, device="cuda"):
    """A zeroed workspace (its status header starts cleared)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def dsa_fold(seqs, ia, u_out, s_row_out, ws):
    _check(_lib.dsa_fold(ctypes.byref(seqs.c), ctypes.byref(ia), _ptr(u_out), _ptr(s_row_out), _ptr(ws), ws.numel(),
                         _stream()), "dsa_fold")


def dsa_index_scores(seqs, ia, row_begin, row_count, scores, ws):
    _check(_lib.dsa_index_scores(ctypes.byref(seqs.c), ctypes.byref(ia), row_begin, row_count, _ptr(scores),
                                 scores.stride(0), _ptr(ws), ws.numel(), _stream()), "dsa_index_scores")


def dsa_topk(seqs, scores, row_begin, row_count, k, idx, ws):
    _check(_lib.dsa_topk(ctypes.byref(seqs.c), _ptr(scores), scores.stride(0), row_begin, row_count, k, _ptr(idx),
                         idx.stride(0), _ptr(ws), ws.numel(), _stream()), "dsa_topk")


def dsa_sparse_attn(seqs, aa, idx, k_sel, ws):
    _check(_lib.dsa_sparse_attn(ctypes.byref(seqs.c), ctypes.byref(aa), _ptr(idx), idx.stride(0), k_sel, _ptr(ws),
                                ws.numel(), _stream()), "dsa_sparse_attn")


def dsa_sparse_attn_bwd(seqs, aa, idx, k_sel, d_out, d_q, d_k, d_v, ws):
    """Backward of dsa_sparse_attn.  aa is the forward's attn_args (its out
    and lse hold the forward's results; lse is required).  d_out [T,H,dv]
    has q's dtype; d_q [T,H,dk] float32 is written; d_k [Tk,>=dk] and d_v
    [Tk,>=dv] float32 accumulate (zero them first; d_v may be a view of d_k's
    first dv columns for the MLA-tied gradient)."""
    _check(_lib.dsa_sparse_attn_bwd(ctypes.byref(seqs.c), ctypes.byref(aa), _ptr(idx), idx.stride(0), k_sel,
                                    _ptr(d_out), d_out.stride(0), d_out.stride(1), _ptr(d_q), d_q.stride(0),
                                    d_q.stride(1), _ptr(d_k), d_k.stride(0), _ptr(d_v), d_v.stride(0), _ptr(ws),
                                    ws.numel(), _stream()), "dsa_sparse_attn_bwd")


def dsa_attn_target(seqs, aa, idx, k_sel, p, ws):
    """Head-averaged attention probabilities of the selected keys (the
    indexer's KL target).  aa is the forward's attn_args (lse required);
    p float32 [T, >= k_sel] is zeroed and written."""
    _check(_lib.dsa_attn_target(ctypes.byref(seqs.c), ctypes.byref(aa), _ptr(idx), idx.stride(0), k_sel, _ptr(p),
                                p.stride(0), _ptr(ws), ws.numel(), _stream()), "dsa_attn_target")


def dsa_indexer_kl(seqs, q_idx, W, k_idx, idx, k_sel, p, loss, d_q, d_W, d_k, ws):
    """The indexer's KL loss over the selection and its gradients (float32
    tensors: q_idx [T,128], W [128,128], k_idx [Tk,128], p [T,>=k_sel];
    loss [T] or None; d_q written; d_W, d_k accumulated)."""
    _check(_lib.dsa_indexer_kl(ctypes.byref(seqs.c), _ptr(q_idx), q_idx.stride(0), _ptr(W), _ptr(k_idx),
                               k_idx.stride(0), _ptr(idx), idx.stride(0), k_sel, _ptr(p), p.stride(0), _ptr(loss),
                               _ptr(d_q), d_q.stride(0), _ptr(d_W), _ptr(d_k), d_k.stride(0), _ptr(ws), ws.numel(),
                               _stream()), "dsa_indexer_kl")


def dsa_forward_host(seqs, ia, aa, k, idx_out, ws, h2d_stream=None, d2h_stream=None):
    """dsa_forward with aa's q and out in pinned host memory (see attn_args);
    the copies run on h2d_stream / d2h_stream (torch.cuda.Stream or None for
    the current stream), the compute on the current stream."""
    cur = _stream()
    sh = ctypes.c_void_p(h2d_stream.cuda_stream) if h2d_stream is not None else cur
    sd = ctypes.c_void_p(d2h_stream.cuda_stream) if d2h_stream is not None else cur
    _check(_lib.dsa_forward_host(ctypes.byref(seqs.c), ctypes.byref(ia), ctypes.byref(aa), k, _ptr(idx_out),
                                 idx_out.stride(0) if idx_out is not None else 0, _ptr(ws), ws.numel(), cur, sh, sd),
           "dsa_forward_host")


def dsa_forward(seqs, ia, aa, k, idx_out, ws):
    _check(_lib.dsa_forward(ctypes.byref(seqs.c), ctypes.byref(ia), ctypes.byref(aa), k, _ptr(idx_out),
                            idx_out.stride(0) if idx_out is not None else 0, _ptr(ws), ws.numel(), _stream()),
           "dsa_forward")


def dsa_select(seqs, ia, k, idx, ws):
    _check(_lib.dsa_select(ctypes.byref(seqs.c), ctypes.byref(ia), k, _ptr(idx), idx.stride(0), _ptr(ws), ws.numel(),
                           _stream()), "dsa_select")


def dsa_select_noalloc(seqs, ia, k, idx):
    """dsa_select without a workspace (for callers that cannot allocate device
    memory): synchronous, returns nothing, raises DsaError on any status."""
    _check(_lib.dsa_select_noalloc(ctypes.byref(seqs.c), ctypes.byref(ia), k, _ptr(idx), idx.stride(0), _stream()),
           "dsa_select_noalloc")


def _need(ok, what):
    if not ok:
        raise ValueError(what)


_DTYPES = {torch.bfloat16: DSA_BF16, torch.float32: DSA_F32}


def _dtype(t):
    _need(t.dtype in _DTYPES, "bfloat16 or float32 expected")
    return _DTYPES[t.dtype]


def _here(seqs, *tensors):
    """Refuse tensors, and a batch's lengths, of another device than the current
    one, whose stream the call would use."""
    dev = tensors[0].get_device()  # (-1: not a CUDA tensor)
    if dev >= 0 and dev == _device() and seqs._index == dev:
        for t in tensors:
            if t.get_device() != dev:
                break
        else:
            return dev
    raise ValueError("tensors and lengths must be on the current CUDA device")


def rope_table(positions, dim, base=10000.0, device="cuda"):
    """cos | sin [positions, dim] (float32) of pos / base^(2i/dim), with the
    angles in 64 bits: a plan-time table for row_args (any other angles will do)."""
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def row_args(norm_dim=0, weight=None, eps=1e-6, rope_begin=0, rope_dim=0, cos_sin=None, interleaved=True):
    """The per-row transform of queries and keys: RMS norm of the columns
    [0, norm_dim) (weight: float32 [norm_dim] or None for ones), then the rotation
    of [rope_begin, rope_begin + rope_dim) by the position's row of cos_sin
    (float32 [positions, rope_dim], cosines then sines); pairs (2i, 2i+1) when
    interleaved, else (i, i + rope_dim/2)."""
    if weight is not None:
        _need(weight.dtype == torch.float32 and weight.is_contiguous() and weight.numel() == norm_dim,
              "weight: contiguous float32 [norm_dim]")
    if rope_dim:
        _need(cos_sin is not None and cos_sin.dtype == torch.float32 and cos_sin.is_contiguous() and cos_sin.dim() == 2
              and cos_sin.shape[1] == rope_dim, "cos_sin: contiguous float32 [positions, rope_dim]")
    a = dsa_row_args(norm_dim, eps, weight.data_ptr() if weight is not None else None, rope_begin, rope_dim,
                     int(interleaved), cos_sin.data_ptr() if rope_dim else None, cos_sin.shape[0] if rope_dim else 0)
    a._keep = (weight, cos_sin)
    devices = {t.device for t in (weight, cos_sin if rope_dim else None) if t is not None}
    _need(len(devices) <= 1, "weight and cos_sin are on one device")
    a._device = devices.pop() if devices else None
    a._index = (weight if weight is not None else cos_sin).get_device() if a._device is not None else None
    return a


def _pool_row(p):
    """Elements between the rows of a page (any, in pages of one row)."""
    return p.stride(1) if p.shape[1] > 1 else p.shape[2]


class Pages:
    """A page table and its pools: table int32 [batch, pages per sequence];
    kv [num_pages, page_size, >=dk], v (its own pool, or None), idx [num_pages,
    page_size, 128] (uint8 e4m3 codes or float32), idx_scale float32 [num_pages,
    page_size].  Pools may be strided by page; keeps the tensors alive."""

    def __init__(self, table, kv=None, v=None, idx=None, idx_scale=None):
        _need(table.dtype == torch.int32 and table.dim() == 2 and table.stride(1) == 1, "table: int32 [batch, n]")
        pools = [p for p in (kv, v, idx, idx_scale) if p is not None]
        _need(pools, "a page table needs a pool")
        n, size = pools[0].shape[:2]
        for p in pools:
            _need(p.shape[0] == n and p.shape[1] == size, "pools of one table have the same pages")
            _need(p.device == table.device, "pools and table are on one device")
        for p in (kv, v):
            _need(p is None or (p.dim() == 3 and p.stride(2) == 1), "kv: [pages, page_size, columns]")
            _need(p is None or p.dtype in (torch.bfloat16, torch.float32), "kv: bfloat16 or float32")
        _need(kv is None or v is None or kv.dtype == v.dtype, "kv and v have one type")
        _need(idx is None or (idx.dim() == 3 and idx.shape[2] == 128 and idx.stride(2) == 1
                              and (idx.stride(1) == 128 or size == 1)
                              and idx.dtype in (torch.uint8, torch.float32)),
              "idx: uint8 or float32 [pages, page_size, 128], rows contiguous")
        _need(idx_scale is None or (idx_scale.dim() == 2 and idx_scale.dtype == torch.float32
                                    and (idx_scale.stride(1) == 1 or size == 1)), "idx_scale: float32 [pages, page_size]")
        self.table, self.kv, self.v, self.idx, self.idx_scale = table, kv, v, idx, idx_scale
        self.batch, self.positions = table.shape[0], table.shape[1] * size

        def page(p):  # (any, in a pool of one page)
            if p is None or n > 1:
                return 0 if p is None else p.stride(0)
            return size * (_pool_row(p) if p.dim() == 3 else 1)

        self.c = dsa_pages(size, n, table.data_ptr(), max(table.stride(0), table.shape[1]) if table.shape[0] == 1 else
                           table.stride(0), page(kv), page(v), page(idx), page(idx_scale))

    def need(self, c):
        """Refuse a batch (a dsa_seqs) that the table does not hold."""
        if self.batch < c.batch or self.positions < c.max_seqlen_k:
            raise ValueError("the table has a row per sequence and an entry per page of the longest")


def append_args(pages, kv_new=None, kv_row=None, idx_new=None, idx_row=None):
    """Rows to append to the pools of `pages`: kv_new [T, dim] (of the KV pool's
    type) and / or idx_new [T, 128], each with its row_args or None."""
    _need(kv_new is not None or idx_new is not None, "nothing to append")
    for t in kv_new, idx_new:
        _need(t is None or t.device == pages.table.device, "new rows are on the pools' device")
    for r in kv_row, idx_row:
        _need(r is None or r._device in (None, pages.table.device), "the rows' weight and cos_sin are on the pools' device")
    a = dsa_append_args()
    a.dtype = _dtype(kv_new if kv_new is not None else idx_new)
    if kv_new is not None:
        _need(pages.kv is not None and kv_new.dtype == pages.kv.dtype, "kv_new has the KV pool's type")
        _need(kv_new.dim() == 2 and kv_new.stride(1) == 1 and kv_new.shape[1] <= pages.kv.shape[2], "kv_new: [T, dim]")
        a.dim, a.kv_new = kv_new.shape[1], kv_new.data_ptr()
        a.kv_new_stride = kv_new.stride(0) if kv_new.shape[0] > 1 else a.dim
        a.kv, a.kv_stride = pages.kv.data_ptr(), _pool_row(pages.kv)
        a.kv_row = ctypes.pointer(kv_row) if kv_row is not None else None
    if idx_new is not None:
        _need(pages.idx is not None and _dtype(idx_new) == a.dtype, "idx_new has kv_new's type")
        _need(idx_new.dim() == 2 and idx_new.stride(1) == 1 and idx_new.shape[1] == 128, "idx_new: [T, 128]")
        a.idx_dtype = DSA_E4M3 if pages.idx.dtype == torch.uint8 else DSA_F32
        a.idx_new, a.idx = idx_new.data_ptr(), pages.idx.data_ptr()
        a.idx_new_stride = idx_new.stride(0) if idx_new.shape[0] > 1 else 128
        a.idx_scale = pages.idx_scale.data_ptr() if pages.idx_scale is not None else None
        a.idx_row = ctypes.pointer(idx_row) if idx_row is not None else None
    a._keep = (pages, kv_new, kv_row, idx_new, idx_row)
    a._rows = min(t.shape[0] for t in (kv_new, idx_new) if t is not None)
    return a


def paged_attn_args(pages, q, scale, out, lse=None):
    """attn_args over the pools of `pages`: q [T,H,dk], out [T,H,dv]; V is the V
    pool, or the first dv columns of the KV rows where there is none."""
    kv, v = pages.kv, pages.v if pages.v is not None else pages.kv
    _need(kv is not None and q.dtype == kv.dtype and out.dtype == q.dtype, "q, out and the KV pool have one type")
    _need(q.shape[2] <= kv.shape[2] and out.shape[2] <= v.shape[2] and q.shape[:2] == out.shape[:2], "q [T,H,dk], out [T,H,dv]")
    _need(q.stride(2) == 1 and out.stride(2) == 1, "q and out: contiguous rows")
    _need(all(t is None or t.device == kv.device for t in (q, out, lse)), "q, out and lse are on the pools' device")
    _need(lse is None or (lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == q.shape[:2]),
          "lse: contiguous float32 [T,H]")
    a = dsa_attn_args(_dtype(q), q.shape[1], q.shape[2], out.shape[2], q.data_ptr(), *_row_strides(q.shape, q.stride()),
                      kv.data_ptr(), _pool_row(kv), v.data_ptr(), _pool_row(v), float(scale), out.data_ptr(),
                      *_row_strides(out.shape, out.stride()), lse.data_ptr() if lse is not None else None)
    a._keep = (pages, q, out, lse)
    a._rows = q.shape[0]
    return a


def _row_strides(shape, s):
    """Token and head strides of rows [T, heads, dim]; a dimension of one, whose
    stride torch leaves open, gets that of rows one after the other."""
    head = s[1] if shape[1] > 1 else shape[2]
    return s[0] if shape[0] > 1 else shape[1] * max(head, shape[2]), head


def _rows_of(seqs, t, shape, dtype):
    s = t.stride()
    if t.shape != shape or len(s) != 3 or shape[0] < seqs.c.total_q or (s[2] != 1 and shape[2] > 1) or t.dtype != dtype:
        raise ValueError("rows: [T, heads, dim] of one shape and type, contiguous columns")
    head = s[1] if shape[1] > 1 else shape[2]  # (as _row_strides, without a call)
    return t.data_ptr(), s[0] if shape[0] > 1 else shape[1] * max(head, shape[2]), head


def dsa_norm_rope(seqs, ra, x, y, ws):
    """y[t,h,:] = the transform ra (row_args or None) of x[t,h,:] at token t's
    position; x, y [T,H,dim] bfloat16 or float32 (y may be x)."""
    dev = _here(seqs, x, y, ws)
    _need(ra is None or ra._index is None or ra._index == dev, "weight and cos_sin are on x's device")
    sh, dt = x.shape, x.dtype
    xp, xt, xh = _rows_of(seqs, x, sh, dt)
    yp, yt, yh = _rows_of(seqs, y, sh, dt)
    _check(_lib.dsa_norm_rope(ctypes.byref(seqs.c), ctypes.byref(ra) if ra is not None else None, _DTYPES.get(dt, -1),
                              sh[1], sh[2], xp, xt, xh, yp, yt, yh, ws.data_ptr(), ws.numel(), _stream()),
           "dsa_norm_rope")


def dsa_norm_rope_bwd(seqs, ra, x, d_y, d_x, d_weight, ws):
    """Backward of dsa_norm_rope: d_x [T,H,dim] (x's type) and d_weight (float32
    [norm_dim] or None) are written from x (None without a norm) and d_y.  ws of
    dsa_workspace_size(DSA_OP_NORM_ROPE_BWD, seqs, norm_dim) bytes."""
    dev = _here(seqs, *[t for t in (x, d_y, d_x, d_weight, ws) if t is not None])
    _need(ra is None or ra._index is None or ra._index == dev, "weight and cos_sin are on x's device")
    sh, dt = d_y.shape, d_y.dtype
    xp, xt, xh = _rows_of(seqs, x, sh, dt) if x is not None else (None, sh[1] * sh[2], sh[2])
    gp, gt, gh = _rows_of(seqs, d_y, sh, dt)
    dp, dt_, dh = _rows_of(seqs, d_x, sh, dt)
    _need(d_weight is None or (d_weight.dtype == torch.float32 and d_weight.is_contiguous()
                               and d_weight.numel() == (ra.norm_dim if ra is not None else 0)),
          "d_weight: contiguous float32 [norm_dim]")
    _check(_lib.dsa_norm_rope_bwd(ctypes.byref(seqs.c), ctypes.byref(ra) if ra is not None else None, _DTYPES.get(dt, -1),
                                  sh[1], sh[2], xp, xt, xh, gp, gt, gh, dp, dt_, dh, _ptr(d_weight), ws.data_ptr(),
                                  ws.numel(), _stream()), "dsa_norm_rope_bwd")


def dsa_cache_append(seqs, pages, ap, ws):
    """Append the queries' tokens (append_args) to the paged cache at their
    positions.  seqs holds the lengths after the append."""
    _here(seqs, pages.table, ws)
    c = seqs.c
    pages.need(c)
    _need(ap._rows >= c.total_q and ap._keep[0] is pages, "a row per query token, appended to these pages")
    _check(_lib.dsa_cache_append(ctypes.byref(c), ctypes.byref(pages.c), ctypes.byref(ap), ws.data_ptr(), ws.numel(),
                                 _stream()), "dsa_cache_append")


def dsa_paged_scores(seqs, pages, u, s_row, row_begin, row_count, scores, ws):
    """Indexer scores of folded queries (u, s_row from dsa_fold) over the paged
    indexer keys; scores float32 [row_count, >= max_seqlen_k], rows one after the
    other, -inf past a row's position.  dsa_topk selects from them."""
    _here(seqs, u, scores, pages.table, ws)
    _need(s_row is None or (s_row.device == u.device and s_row.dtype == torch.float32 and s_row.is_contiguous()
                            and s_row.numel() >= seqs.c.total_q), "s_row: contiguous float32 [T]")
    c, dt, us, (rows, cols), st = seqs.c, u.dtype, u.shape, scores.shape, scores.stride()
    pages.need(c)
    _need(pages.idx is not None, "an indexer-key pool")
    _need(dt == pages.idx.dtype and u.is_contiguous() and us[0] >= c.total_q and us[1] == 128,
          "u: contiguous [T, 128] of the pool's type")
    _need(scores.dtype == torch.float32 and (st[1] == 1 or cols == 1) and rows >= row_count and cols >= c.max_seqlen_k,
          "scores: float32 [row_count, >= max_seqlen_k]")
    # (the -inf behind a row fills it up to the next row: columns beside a view are not this call's)
    _need(row_count <= 1 or st[0] == cols, "scores: rows one after the other")
    fp8 = dt == torch.uint8
    _check(_lib.dsa_paged_scores(ctypes.byref(c), ctypes.byref(pages.c), DSA_E4M3 if fp8 else DSA_F32, u.data_ptr(),
                                 _ptr(s_row), pages.idx.data_ptr(), _ptr(pages.idx_scale) if fp8 else None, row_begin,
                                 row_count, scores.data_ptr(), cols, ws.data_ptr(), ws.numel(),
                                 _stream()), "dsa_paged_scores")


def paged_indexer_args(pages, q_idx, q_idx_scale, w_index, k_per_row=None):
    """indexer_args over the indexer-key pool of `pages`: q_idx [T, 128] of the
    pool's type, with q_idx_scale float32 [T] and a bfloat16 w_index [128, 128] for
    codes, None and a float32 one for float32; k_per_row int32 [T] or None."""
    _need(pages.idx is not None and pages.idx.dtype == q_idx.dtype, "q_idx has the indexer-key pool's type")
    _need(q_idx.dim() == 2 and q_idx.shape[1] == 128 and q_idx.is_contiguous(), "q_idx: contiguous [T, 128]")
    fp8, rows = q_idx.dtype == torch.uint8, q_idx.shape[0]
    _need(w_index.dtype == (torch.bfloat16 if fp8 else torch.float32) and w_index.shape == (128, 128)
          and w_index.is_contiguous(), "w_index: contiguous [128, 128], bfloat16 for codes, else float32")
    _need((q_idx_scale is not None) == fp8, "q_idx_scale: for codes")
    for t, dt in (q_idx_scale, torch.float32), (k_per_row, torch.int32):
        _need(t is None or (t.dtype == dt and t.is_contiguous() and t.numel() >= rows),
              "q_idx_scale: contiguous float32 [T], k_per_row: contiguous int32 [T]")
    _need(all(t is None or t.device == pages.idx.device for t in (q_idx, q_idx_scale, w_index, k_per_row)),
          "queries, weights and k_per_row are on the pools' device")
    return indexer_args(q_idx, q_idx_scale, w_index, pages.idx, pages.idx_scale if q_idx.dtype == torch.uint8 else None,
                        k_per_row)


def dsa_paged_select(seqs, pages, ia, k, idx, ws):
    """dsa_select over the paged indexer keys (ia from paged_indexer_args).  ws
    of dsa_workspace_size(DSA_OP_PAGED_SELECT, seqs, k, ia) bytes."""
    _here(seqs, idx, pages.table, ws)
    pages.need(seqs.c)
    _need(pages.idx is not None and (ia.k_idx or 0) == pages.idx.data_ptr()
          and (not ia.k_idx_scale or (pages.idx_scale is not None and ia.k_idx_scale == pages.idx_scale.data_ptr())),
          "arguments over these pages")
    _need(ia._keep[0].shape[0] >= seqs.total_q, "a q_idx row per query token")
    _need(idx.dtype == torch.int32 and idx.shape[0] >= seqs.total_q
          and idx.shape[1] >= k and idx.stride(1) == 1, "idx: int32 [T, >= k]")
    _check(_lib.dsa_paged_select(ctypes.byref(seqs.c), ctypes.byref(pages.c), ctypes.byref(ia), k, _ptr(idx),
                                 idx.stride(0) if idx.shape[0] > 1 else idx.shape[1], _ptr(ws), ws.numel(), _stream()),
           "dsa_paged_select")


def dsa_paged_attn(seqs, pages, aa, idx, k_sel, ws):
    """Attention of the queries over the paged KV rows (aa from
    paged_attn_args): dense causal with idx None and k_sel 0, else over idx
    int32 [T, >= k_sel] of local positions (-1 unused).  ws of
    dsa_workspace_size(DSA_OP_PAGED_ATTN, seqs, k_sel, None, aa) bytes."""
    _here(seqs, pages.table, ws)
    c = seqs.c
    pages.need(c)
    _need(aa._rows >= c.total_q and aa._keep[0] is pages, "a q row per token, arguments over these pages")
    ip, ld = None, 0
    if idx is not None:
        (rows, cols), st = idx.shape, idx.stride()
        _here(seqs, idx)
        _need(idx.dtype == torch.int32 and rows >= c.total_q and (st[1] == 1 or cols == 1) and cols >= k_sel,
              "idx: int32 [T, >= k_sel]")
        ip, ld = idx.data_ptr(), st[0] if rows > 1 else max(cols, k_sel)
    _check(_lib.dsa_paged_attn(ctypes.byref(c), ctypes.byref(pages.c), ctypes.byref(aa), ip, ld, k_sel, ws.data_ptr(),
                               ws.numel(), _stream()), "dsa_paged_attn")


def dsa_sync_status(ws):
    """Synchronise the current stream; return (status, detail) recorded on the
    device since the last call, and clear it."""
    d = _I64(0)
    code = _lib.dsa_sync_status(_ptr(ws), _stream(), ctypes.byref(d))
    return code, d.value


def check_device_status(ws, where="device"):
    code, detail = dsa_sync_status(ws)
    if code != DSA_OK:
        raise DsaError(code, where, detail)


def dsa_selftest_wait_timeout(ws, budget_cycles):
    _check(_lib.dsa_selftest_wait_timeout(_ptr(ws), ws.numel(), budget_cycles, _stream()), "dsa_selftest_wait_timeout")


def raw_call(name, *args):
    """Call a C entry point with raw ctypes arguments (tests of the ABI)."""
    return getattr(_lib, name)(*args)
