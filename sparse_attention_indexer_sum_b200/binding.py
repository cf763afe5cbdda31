"""ctypes binding of libic_b200.so (include/ic.h), one Python function per C entry point.

Argument marshalling only: shapes are read off the torch tensors, pointers and
the current CUDA stream are handed to the library, and a non-zero status
raises ``ICError``.  Every step of the path runs in the library's kernels;
there is no fallback of any kind: if the library is missing the first call
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# IC_DEBUG_BOUNDS=1 in the environment selects the debug-bounds build of the same
# library (device-side index checks reported as IC_ERR_BOUNDS; see ic.h)
LIB_PATH = os.path.join(_PKG, "libic_b200_debug.so" if os.environ.get("IC_DEBUG_BOUNDS") == "1"
                        else "libic_b200.so")

IC_OK = 0
IC_ERR_INVALID_ARG = -1
IC_ERR_UNSUPPORTED = -2
IC_ERR_WORKSPACE = -3
IC_ERR_CUDA = -4
IC_ERR_TIMEOUT = -5
IC_ERR_BOUNDS = -6
IC_F32, IC_BF16, IC_E4M3, IC_MXF4 = 0, 1, 2, 3

# names declared in include/ic.h (checked against the header by the tests)
EXPORTS = ("ic_last_error", "ic_version", "ic_device_status", "ic_trace_begin", "ic_trace_end",
           "ic_quant_e4m3_rows", "ic_pack_kv_e4m3",
           "ic_indexer_scores", "ic_indexer_topk", "ic_indexer_topk_workspace_size", "ic_topk",
           "ic_topk_varlen", "ic_sparse_attn",
           "ic_attn_workspace_size",
           "ic_layer_stack", "ic_decode_step", "ic_stack_workspace_size",
           "ic_sparse_attn_noalloc", "ic_layer_stack_rows", "ic_layer_stack_varlen",
           "ic_rms_norm", "ic_cache_append", "ic_indexer_scores_paged", "ic_sparse_attn_paged",
           "ic_decode_step_paged")


class ICError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("ic status %d: %s" % (status, msg))
        self.status = status


class ic_layer_io(ctypes.Structure):
    _fields_ = [("q_idx", ctypes.c_void_p), ("q_scale", ctypes.c_void_p),
                ("k_idx", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("q", ctypes.c_void_p), ("kv", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class ic_stack_desc(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("batch", ctypes.c_int), ("decode", ctypes.c_int),
                ("k", ctypes.c_int), ("idx_dtype", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("attn_dtype", ctypes.c_int), ("heads", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("ld_kv", ctypes.c_long),
                ("scale", ctypes.c_float), ("flags", ctypes.c_int)]


class ic_paging(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("ld_table", ctypes.c_long),
                ("max_pages", ctypes.c_int), ("seq_lens", ctypes.c_void_p),
                ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int)]


IC_STACK_FUSED_TOPK = 1
IC_ROPE_KV_HALVES, IC_ROPE_K_HALVES = 1, 2


_lib = None


def lib() -> ctypes.CDLL:
    """Opens libic_b200.so (built in-tree by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libic_b200.so is not built (%s); run "
                           "`python -m sparse_attention_indexer_sum_b200.build`" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, I, Lg, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_float, ctypes.c_size_t
    L.ic_last_error.restype = ctypes.c_char_p
    L.ic_last_error.argtypes = []
    L.ic_version.restype = I
    L.ic_device_status.argtypes = [P]
    L.ic_trace_begin.argtypes = [P, I]
    L.ic_trace_begin.restype = I
    L.ic_trace_end.argtypes = [P, P, P, I]
    L.ic_trace_end.restype = Lg
    L.ic_quant_e4m3_rows.argtypes = [P, I, Lg, I, P, P, P]
    L.ic_pack_kv_e4m3.argtypes = [P, Lg, Lg, P, Lg, P]
    L.ic_indexer_scores.argtypes = [P, P, P, P, P, I, I, I, I, I, I, Lg, P, Lg, P]
    L.ic_indexer_topk.argtypes = [P, P, P, P, P, I, I, I, I, I, Lg, I, P, P, S, P]
    L.ic_indexer_topk_workspace_size.argtypes = [I, I, Lg]
    L.ic_indexer_topk_workspace_size.restype = S
    L.ic_topk.argtypes = [P, Lg, I, Lg, Lg, I, P, P]
    L.ic_topk_varlen.argtypes = [P, Lg, I, Lg, P, I, P, P]
    L.ic_sparse_attn.argtypes = [P, P, Lg, P, P, I, I, I, I, I, I, I, I, F, P, P, P, S, P]
    L.ic_attn_workspace_size.argtypes = [I, I, I, I, I]
    L.ic_attn_workspace_size.restype = S
    L.ic_layer_stack.argtypes = [ctypes.c_char_p, ctypes.POINTER(ic_stack_desc),
                                 ctypes.POINTER(ic_layer_io), I, P, P, S, P]
    L.ic_decode_step.argtypes = L.ic_layer_stack.argtypes
    L.ic_layer_stack_rows.argtypes = [ctypes.c_char_p, ctypes.POINTER(ic_stack_desc),
                                      ctypes.POINTER(ic_layer_io), I, Lg, Lg, P, P, S, P]
    L.ic_layer_stack_varlen.argtypes = [ctypes.c_char_p, ctypes.POINTER(ic_stack_desc),
                                        ctypes.POINTER(ic_layer_io), I, ctypes.POINTER(Lg), I, P,
                                        P, S, P]
    L.ic_stack_workspace_size.argtypes = [ctypes.POINTER(ic_stack_desc)]
    L.ic_stack_workspace_size.restype = S
    L.ic_sparse_attn_noalloc.argtypes = [P, P, Lg, P, P, I, I, I, I, I, I, I, I, F, P, P, P]
    L.ic_rms_norm.argtypes = [P, Lg, P, Lg, I, P, I, F, Lg, I, P, Lg, P, Lg, P, Lg, P, P]
    L.ic_cache_append.argtypes = [Lg, P, P, P, Lg, P, Lg, P, Lg, I, P, Lg, P, P, I, Lg, I, P]
    PG = ctypes.POINTER(ic_paging)
    L.ic_indexer_scores_paged.argtypes = [P, P, P, P, P, I, I, I, I, PG, I, P, Lg, P]
    L.ic_sparse_attn_paged.argtypes = [P, P, Lg, PG, P, I, I, I, I, I, I, I, F, P, P, P, S, P]
    L.ic_decode_step_paged.argtypes = [ctypes.c_char_p, ctypes.POINTER(ic_stack_desc), PG,
                                       ctypes.POINTER(ic_layer_io), I, P, P, S, P]
    for name in ("ic_rms_norm", "ic_cache_append", "ic_indexer_scores_paged",
                 "ic_sparse_attn_paged", "ic_decode_step_paged"):
        getattr(L, name).restype = I
    for name in ("ic_device_status", "ic_quant_e4m3_rows", "ic_pack_kv_e4m3", "ic_indexer_scores",
                 "ic_topk",
                 "ic_topk_varlen", "ic_indexer_topk",
                 "ic_sparse_attn", "ic_layer_stack", "ic_decode_step", "ic_sparse_attn_noalloc",
                 "ic_layer_stack_rows", "ic_layer_stack_varlen"):
        getattr(L, name).restype = I
    _lib = L
    return L


def ic_last_error() -> str:
    return lib().ic_last_error().decode()


def ic_version() -> int:
    return int(lib().ic_version())


def _check(st: int):
    if st != IC_OK:
        raise ICError(st, ic_last_error())


def _p(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return IC_F32
    if t.dtype == torch.bfloat16:
        return IC_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return IC_E4M3
    raise ValueError("unsupported dtype %s" % t.dtype)


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def ic_device_status(stream=None):
    """Synchronises the stream; raises ICError(IC_ERR_TIMEOUT) if a device wait gave up
    (IC_ERR_BOUNDS if a debug-bounds check failed)."""
    _check(lib().ic_device_status(_stream(stream)))


KIND_NAMES = {1: "indexer_tc_bf16", 2: "indexer_tc_e4m3", 3: "indexer_f32", 4: "fill_masked",
              5: "topk", 6: "attn_mla", 7: "attn_combine", 8: "attn_f32", 9: "quant_e4m3",
              10: "topk_merge", 11: "indexer_topk_bf16", 12: "indexer_topk_e4m3",
              13: "attn_mla_kv8", 14: "pack_kv_e4m3", 15: "fill_valid", 16: "rms_norm",
              17: "cache_append", 18: "attn_mla_kv4"}


def ic_trace_begin(capacity: int = 4096, stream=None):
    """Starts per-launch event tracing on this thread (see ic.h)."""
    _check(lib().ic_trace_begin(_stream(stream), int(capacity)))
    return int(capacity)


def ic_trace_end(capacity: int = 4096):
    """Stops tracing; returns (launches, [(kind_name, ms, work), ...])."""
    import numpy as np
    ms = np.zeros(capacity, np.float32)
    kinds = np.zeros(capacity, np.int32)
    work = np.zeros(capacity, np.float64)
    n = lib().ic_trace_end(ms.ctypes.data_as(ctypes.c_void_p), kinds.ctypes.data_as(ctypes.c_void_p),
                           work.ctypes.data_as(ctypes.c_void_p), int(capacity))
    if n < 0:
        raise ICError(int(n), ic_last_error())
    m = min(int(n), capacity)
    return int(n), [(KIND_NAMES.get(int(kinds[i]), str(kinds[i])), float(ms[i]), float(work[i]))
                    for i in range(m)]


def ic_quant_e4m3_rows(x: torch.Tensor, codes=None, scales=None, stream=None):
    """Per-row e4m3 codes (uint8) and fp32 scales of x[..., n]."""
    _contig(x)
    n = x.shape[-1]
    rows = x.numel() // n
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check(lib().ic_quant_e4m3_rows(_p(x), dtype_code(x), rows, n, _p(codes), _p(scales),
                                    _stream(stream)))
    return codes, scales


KV8_ROW_BYTES = 656


def ic_pack_kv_e4m3(kv: torch.Tensor, out=None, stream=None):
    """fp8 latent-KV cache rows [..., 656] uint8 of bf16 latent rows kv [..., 576]
    (512 e4m3 codes in four 128-dim groups, 4 fp32 group scales, 64 bf16 rope dims)."""
    if kv.dtype != torch.bfloat16 or kv.shape[-1] != 576 or kv.stride(-1) != 1:
        raise ValueError("kv must be bf16 [..., 576] with contiguous rows")
    rows = kv.numel() // 576
    if out is None:
        out = torch.empty(kv.shape[:-1] + (KV8_ROW_BYTES,), dtype=torch.uint8, device=kv.device)
    _contig(kv, out)
    _check(lib().ic_pack_kv_e4m3(_p(kv), rows, 576, _p(out), out.shape[-1], _stream(stream)))
    return out


def ic_indexer_scores(q, k, w, scores=None, *, pos0: int = 0, q_scale=None, k_scale=None,
                      stream=None):
    """Indexer scores [B, R, Lk] (or [R, Lk] without a batch axis) of q [B?,R,H,D],
    k [B?,Lk,D], w [B?,R,H]; e4m3 inputs (uint8 codes) take q_scale [B?,R,H], k_scale [B?,Lk]."""
    _contig(q, k, w, q_scale, k_scale)
    squeeze = q.dim() == 3
    B = 1 if squeeze else q.shape[0]
    R, H, D = q.shape[-3:]
    Lk = k.shape[-2]
    if scores is None:
        shape = (R, Lk) if squeeze else (B, R, Lk)
        scores = torch.empty(shape, dtype=torch.float32, device=q.device)
    ld = scores.stride(-2)
    _check(lib().ic_indexer_scores(_p(q), _p(q_scale), _p(k), _p(k_scale), _p(w), dtype_code(q),
                                   B, H, D, R, Lk, int(pos0), _p(scores), ld, _stream(stream)))
    return scores


def ic_indexer_topk_workspace_size(batch: int, Lk: int, pos0: int) -> int:
    return int(lib().ic_indexer_topk_workspace_size(int(batch), int(Lk), int(pos0)))


def ic_indexer_topk(q, k, w, k_top: int, workspace, *, pos0: int, q_scale=None, k_scale=None,
                    idx=None, stream=None):
    """Indexer and top-k in one pass for one query per sequence: q [B,1,H,D],
    k [B,Lk,D], w [B,1,H] (e4m3 codes take q_scale [B,1,H], k_scale [B,Lk]); returns
    idx [B, k_top] int32.  The scores are never written."""
    _contig(q, k, w, q_scale, k_scale)
    if q.dim() != 4 or q.shape[1] != 1:
        raise ValueError("q must be [B, 1, H, D]")
    B, _, H, D = q.shape
    Lk = k.shape[-2]
    if idx is None:
        idx = torch.empty((B, k_top), dtype=torch.int32, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().ic_indexer_topk(_p(q), _p(q_scale), _p(k), _p(k_scale), _p(w), dtype_code(q), B,
                                 H, D, Lk, int(pos0), int(k_top), _p(idx), _p(workspace),
                                 ws_bytes, _stream(stream)))
    return idx


def ic_topk(scores, k: int, *, n: int | None = None, pos0: int = -1, idx=None, stream=None):
    """Exact top-k indices [rows, k] (int32, ascending, -1 padded) of scores [rows, ld].
    pos0 >= 0 makes the rows causal: row r keeps columns s <= pos0 + r."""
    rows = scores.shape[0]
    n = scores.shape[1] if n is None else n
    if scores.stride(1) != 1:
        raise ValueError("scores rows must be contiguous")
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=scores.device)
    _check(lib().ic_topk(_p(scores), rows, n, scores.stride(0), int(pos0), int(k), _p(idx),
                         _stream(stream)))
    return idx


def ic_topk_varlen(scores, k: int, valid_len, *, n: int | None = None, idx=None, stream=None):
    """Exact top-k indices [rows, k] of scores [rows, ld] with row r's candidates the
    columns s < valid_len[r] (device int32 [rows])."""
    rows = scores.shape[0]
    n = scores.shape[1] if n is None else n
    if scores.stride(1) != 1:
        raise ValueError("scores rows must be contiguous")
    if valid_len.dtype != torch.int32 or valid_len.numel() != rows:
        raise ValueError("valid_len must be int32 [rows]")
    _contig(valid_len)
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=scores.device)
    _check(lib().ic_topk_varlen(_p(scores), rows, n, scores.stride(0), _p(valid_len), int(k),
                                _p(idx), _stream(stream)))
    return idx


def ic_attn_workspace_size(batch: int, rows: int, heads: int, dv: int, k: int) -> int:
    return int(lib().ic_attn_workspace_size(batch, rows, heads, dv, k))


def ic_sparse_attn(q, kv, idx, scale: float, *, v=None, dv: int | None = None, out=None, lse=None,
                   workspace=None, stream=None):
    """Sparse attention.  q [B?,R,heads,dk]; kv [B?,Lkv,ld_kv]; idx [B?,R,k];
    v [B?,Lkv,dv] for the MQA form (fp32), else absorbed MLA over kv[..., :dv]: a bf16
    cache, or an fp8 cache (uint8 rows of ic_pack_kv_e4m3) with q and out bf16."""
    _contig(q, idx, v)
    if kv.stride(-1) != 1:
        raise ValueError("kv rows must be contiguous")
    squeeze = q.dim() == 3
    B = 1 if squeeze else q.shape[0]
    R, heads, dk = q.shape[-3:]
    Lkv = kv.shape[-2]
    kk = idx.shape[-1]
    if v is not None:
        dv = v.shape[-1]
    elif dv is None:
        dv = 512
    if out is None:
        out = torch.empty(q.shape[:-1] + (dv,), dtype=q.dtype, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    dt = IC_E4M3 if (v is None and kv.dtype == torch.uint8) else dtype_code(q)
    _check(lib().ic_sparse_attn(_p(q), _p(kv), kv.stride(-2), _p(v), _p(idx), dt, B, R,
                                heads, dk, dv, Lkv, kk, float(scale), _p(out), _p(lse),
                                _p(workspace), ws_bytes, _stream(stream)))
    return out


def ic_sparse_attn_noalloc(q, kv, idx, scale: float, *, out, dv: int = 512, lse=None,
                           stream=None):
    """Absorbed-MLA sparse attention whose split scratch is the library's fixed device
    array rather than a workspace (for callers that cannot allocate; at most
    IC_NOALLOC_MAX_QUERIES = 64 queries).  q [B?,R,16,576] bf16; kv [B?,Lkv,ld_kv];
    idx [B?,R,k] int32.  The caller passes ``out`` [B?,R,16,dv] bf16 (and, if wanted,
    ``lse`` [B?,R,16] f32), both contiguous: this wrapper allocates nothing either.
    Calls that overlap on the GPU race on the shared array."""
    _contig(q, idx, out, lse)
    if kv.stride(-1) != 1:
        raise ValueError("kv rows must be contiguous")
    squeeze = q.dim() == 3
    B = 1 if squeeze else q.shape[0]
    R, heads, dk = q.shape[-3:]
    if idx.dtype != torch.int32 or tuple(idx.shape[:-1]) != tuple(q.shape[:-2]):
        raise ValueError("idx must be int32 [B?, R, k] matching q")
    if out is None or out.dtype != q.dtype or tuple(out.shape) != tuple(q.shape[:-1]) + (dv,):
        raise ValueError("out must be a %s tensor of shape %s" % (
            q.dtype, tuple(q.shape[:-1]) + (dv,)))
    if lse is not None and (lse.dtype != torch.float32 or
                            tuple(lse.shape) != tuple(q.shape[:-1])):
        raise ValueError("lse must be a float32 tensor of shape %s" % (tuple(q.shape[:-1]),))
    _check(lib().ic_sparse_attn_noalloc(_p(q), _p(kv), kv.stride(-2), None, _p(idx),
                                        dtype_code(q), B, R, heads, dk, dv, kv.shape[-2],
                                        idx.shape[-1], float(scale), _p(out), _p(lse),
                                        _stream(stream)))
    return out


def make_desc(*, L, k, H, D, idx_dtype, heads, dk, dv, attn_dtype, scale, ld_kv=None, batch=1,
              decode=False, flags=0) -> ic_stack_desc:
    return ic_stack_desc(L=L, batch=batch, decode=int(bool(decode)), k=k, idx_dtype=idx_dtype, H=H,
                         D=D, attn_dtype=attn_dtype, heads=heads, dk=dk, dv=dv,
                         ld_kv=dk if ld_kv is None else ld_kv, scale=scale, flags=flags)


def ic_stack_workspace_size(desc: ic_stack_desc) -> int:
    return int(lib().ic_stack_workspace_size(ctypes.byref(desc)))


def _layers(layers):
    arr = (ic_layer_io * len(layers))()
    for i, d in enumerate(layers):
        arr[i] = ic_layer_io(*[(d.get(f).data_ptr() if d.get(f) is not None else None)
                               for f, _ in ic_layer_io._fields_])
    return arr


def ic_layer_stack(pattern: str, desc: ic_stack_desc, layers: list[dict], t_cache, workspace,
                   stream=None):
    """Prefill layer stack; layers are dicts with the ic_layer_io field names."""
    arr = _layers(layers)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().ic_layer_stack(pattern.encode(), ctypes.byref(desc), arr, len(layers),
                                _p(t_cache), _p(workspace), ws_bytes, _stream(stream)))


def ic_layer_stack_rows(pattern: str, desc: ic_stack_desc, layers: list[dict], row0: int,
                        rows: int, t_cache, workspace, stream=None):
    """Prefill stack for query rows [row0, row0 + rows) of the desc.L-token sequence.
    Row-indexed layer tensors (q_idx, q_scale, w, q, out, lse) and t_cache hold just
    those rows; k_idx, k_scale and kv hold all desc.L keys."""
    arr = _layers(layers)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().ic_layer_stack_rows(pattern.encode(), ctypes.byref(desc), arr, len(layers),
                                     int(row0), int(rows), _p(t_cache), _p(workspace), ws_bytes,
                                     _stream(stream)))


def ic_layer_stack_varlen(pattern: str, desc: ic_stack_desc, layers: list[dict], cu_seqlens,
                          t_cache, workspace, stream=None):
    """Prefill stack over sequences packed along the row axis; cu_seqlens = [0, L_0,
    L_0 + L_1, ...] (host ints).  Every layer tensor holds the packed rows."""
    cu = (ctypes.c_long * len(cu_seqlens))(*[int(x) for x in cu_seqlens])
    arr = _layers(layers)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().ic_layer_stack_varlen(pattern.encode(), ctypes.byref(desc), arr, len(layers), cu,
                                       len(cu_seqlens) - 1, _p(t_cache), _p(workspace), ws_bytes,
                                       _stream(stream)))


def ic_decode_step(pattern: str, desc: ic_stack_desc, layers: list[dict], t_cache, workspace,
                   stream=None):
    """Decode step over the layer stack (desc.decode = 1)."""
    arr = _layers(layers)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().ic_decode_step(pattern.encode(), ctypes.byref(desc), arr, len(layers),
                                _p(t_cache), _p(workspace), ws_bytes, _stream(stream)))


def decode_step_graph(pattern: str, desc: ic_stack_desc, layers: list[dict], t_cache, workspace,
                      warmup: int = 1) -> torch.cuda.CUDAGraph:
    """One ic_decode_step captured into a CUDA graph over these buffers.

    ``graph.replay()`` reruns the whole step (its kernels and the programmatic
    launch edges between them) with one launch from the host, on the current
    stream.  Every replay reads the same input tensors and writes the same
    outputs: a caller updates the inputs in place between replays.  The step
    allocates nothing, so the graph holds no memory of its own."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(warmup):  # first-call set-up (kernel attributes) outside the capture
            ic_decode_step(pattern, desc, layers, t_cache, workspace, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    # relaxed: the step's per-launch host calls (kernel attributes, device queries)
    # are not stream work and need not be refused while capturing
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        ic_decode_step(pattern, desc, layers, t_cache, workspace)
    return graph


# ------------------------------------------------------------------ around the path
# These wrappers also run for single tokens, where the host's time per call counts: they
# read each tensor's properties once and pass pointers as plain integers.
KV4_ROW_BYTES = 400
_DT = {torch.float32: IC_F32, torch.bfloat16: IC_BF16}
_KV_ROW = {IC_BF16: 2 * 576, IC_E4M3: KV8_ROW_BYTES, IC_MXF4: KV4_ROW_BYTES}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _one_device(first, *ts) -> int:
    """The index of the CUDA device that every given tensor lives on (else a ValueError)."""
    dev = first.get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            break
    else:
        if dev >= 0:
            return dev
        t = first
    bad = [str(u.device) for u in (first, t) if u.get_device() < 0]
    if bad:
        raise ValueError("tensors must be on a CUDA device (got one on %s)" % bad[0])
    raise ValueError("tensors are on cuda:%d and cuda:%d" % (dev, t.get_device()))


class _On:
    """Makes device `dev` current and `stream` the one that allocations are made for; yields
    the raw stream to launch on."""

    def __init__(self, dev: int, stream):
        self.dev, self.stream, self.held = dev, stream, []

    def __enter__(self):
        if self.dev != torch.cuda.current_device():
            self.held.append(torch.cuda.device(self.dev))
            self.held[-1].__enter__()
        s = self.stream
        if s is None:
            return torch.cuda.current_stream().cuda_stream
        if not isinstance(s, torch.cuda.Stream):
            s = torch.cuda.ExternalStream(int(s), device=self.dev)
        elif s.device.index != self.dev:
            self.__exit__(None, None, None)
            raise ValueError("stream of %s, tensors on cuda:%d" % (s.device, self.dev))
        self.held.append(torch.cuda.stream(s))
        self.held[-1].__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        while self.held:
            self.held.pop().__exit__(*exc)


def _rows2d(t, name, n, dtype):
    """(rows, row stride) of t [..., n] whose leading dims are evenly spaced."""
    if t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    shape = t.shape
    if not shape or shape[-1] != n:
        raise ValueError("%s must be [..., %d]" % (name, n))
    if t.is_contiguous():
        return t.numel() // n if n else 0, n
    stride = t.stride()
    if n > 1 and stride[-1] != 1:
        raise ValueError("%s rows must be contiguous" % name)
    rows, ld = 1, None
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] != 1:
            if ld is None:
                ld = stride[i]
            elif stride[i] != ld * rows:
                raise ValueError("%s rows must be evenly spaced" % name)
            rows *= shape[i]
    return rows, n if ld is None else ld


def _like(t, name, shape, dtype):
    """The row stride of t, which has the given shape."""
    if t.shape != shape:
        raise ValueError("%s must have x's shape" % name)
    if t.dtype == dtype and t.is_contiguous():
        return shape[-1]
    return _rows2d(t, name, shape[-1], dtype)[1]


def _pool(t, name, dtype, row_bytes=0):
    """(slots, row stride in elements) of a cache [slots, w] or [pages, page_size, w]."""
    shape = t.shape
    if len(shape) not in (2, 3):
        raise ValueError("%s must be [slots, width] or [pages, page_size, width]" % name)
    w = shape[-1]
    if w * t.element_size() < row_bytes:
        raise ValueError("%s rows must hold %d bytes" % (name, row_bytes))
    if w and t.dtype == dtype and t.is_contiguous():
        return t.numel() // w, w
    return _rows2d(t, name, w, dtype)


def _kv_pool(kv_cache, kv_dtype):
    if kv_dtype is None and kv_cache.dtype == torch.bfloat16:
        kv_dtype = IC_BF16
    if kv_dtype not in _KV_ROW:
        raise ValueError("kv_dtype must be IC_BF16, IC_E4M3 or IC_MXF4")
    slots, ld = _pool(kv_cache, "kv_cache", torch.bfloat16 if kv_dtype == IC_BF16 else torch.uint8,
                      _KV_ROW[kv_dtype])
    return kv_dtype, slots, ld


def _launch(dev, stream, call, *args):
    """call(*args, raw stream) with `dev` current; its status is checked."""
    # the raw getters take a tenth of the time of current_device() and current_stream()
    if stream is None and dev == torch._C._cuda_getDevice():
        st = call(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with _On(dev, stream) as raw:
            st = call(*args, raw)
    if st != IC_OK:
        raise ICError(st, ic_last_error())


def _new(shape, dtype, dev, stream):
    """A new tensor on device `dev`, allocated for `stream`."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    with _On(dev, stream):
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))


def ic_rms_norm(x, weight, eps: float = 1e-6, *, residual=None, h=None, y=None, codes=None,
                scales=None, stream=None):
    """RMS norm of x [..., n] (+ residual): h = x + residual, y = h / sqrt(mean h^2 + eps) *
    weight.  Writes the outputs that are given (h, y like x; codes uint8 [..., n] with
    scales f32 [..., ceil(n / 128)]), or a new y if none is; returns (y, codes, scales)."""
    dt, shape = x.dtype, x.shape
    if dt not in _DT or not shape:
        raise ValueError("x must be bf16 or fp32 [..., n]")
    n = shape[-1]
    rows, ld_x = _rows2d(x, "x", n, dt)
    if weight.dtype not in _DT or weight.dim() != 1 or weight.numel() != n or \
            not weight.is_contiguous():
        raise ValueError("weight must be bf16 or fp32 [%d], contiguous" % n)
    dev = _one_device(x, weight, residual, h, y, codes, scales)
    if h is None and y is None and codes is None:
        y = _new(shape, dt, dev, stream)
    ld_r = ld_h = ld_y = ld_c = 0
    if residual is not None:
        ld_r = _like(residual, "residual", shape, dt)
    if h is not None:
        ld_h = _like(h, "h", shape, dt)
    if y is not None:
        ld_y = _like(y, "y", shape, dt)
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales go together")
    if codes is not None:
        ld_c = _like(codes, "codes", shape, torch.uint8)
        if scales.dtype != torch.float32 or not scales.is_contiguous() or \
                scales.shape != shape[:-1] + (-(-n // 128),):
            raise ValueError("scales must be fp32 [..., %d], contiguous" % -(-n // 128))
    if rows == 0:
        return y, codes, scales
    _launch(dev, stream, lib().ic_rms_norm,
            x.data_ptr(), ld_x, _ptr(residual), ld_r, _DT[dt], weight.data_ptr(),
            _DT[weight.dtype], eps, rows, n, _ptr(h), ld_h, _ptr(y), ld_y, _ptr(codes), ld_c,
            _ptr(scales))
    return y, codes, scales


def rope_table(positions: int, theta: float = 10000.0, device=None) -> torch.Tensor:
    """cos | sin [positions, 64] f32 of position * theta^(-i / 32), i = 0..31, for
    ic_cache_append; the angles are taken in 64 bits, so far positions keep theirs."""
    inv = float(theta) ** (-torch.arange(32, dtype=torch.float64, device=device) / 32)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def ic_cache_append(slots, *, kv=None, kv_cache=None, kv_dtype=None, k=None, k_cache=None,
                    k_scale=None, pos=None, rope=None, kv_halves: bool = False,
                    k_halves: bool = False, stream=None):
    """Writes the latent rows kv [rows, 576] and / or the indexer keys k [rows, 128] (bf16)
    of `rows` tokens to rows slots [rows] (int64; negative: not written) of kv_cache
    ([slots, w] or [pages, page_size, w]; kv_dtype IC_BF16, IC_E4M3 or IC_MXF4) and k_cache
    (bf16, or uint8 e4m3 codes with k_scale), rotated by rope [P, 64] at positions pos."""
    if slots.dtype != torch.int64 or slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError("slots must be int64 [rows], contiguous")
    rows = slots.numel()
    dev = _one_device(slots, kv, kv_cache, k, k_cache, k_scale, pos, rope)
    if (kv is None) != (kv_cache is None) or (k is None) != (k_cache is None):
        raise ValueError("kv goes with kv_cache, k with k_cache")
    if kv is None and k is None:
        raise ValueError("nothing to append")
    if (rope is None) != (pos is None):
        raise ValueError("rope goes with pos")
    rope_rows = 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 2 or rope.shape[1] != 64 or \
                not rope.is_contiguous():
            raise ValueError("rope must be fp32 [positions, 64], contiguous")
        if pos.dtype != torch.int32 or pos.dim() != 1 or pos.numel() != rows or \
                not pos.is_contiguous():
            raise ValueError("pos must be int32 [rows], contiguous")
        rope_rows = rope.shape[0]
    count = None
    ld_kv = ld_cache = ld_k = 0
    k_dt = IC_BF16
    if kv is not None:
        n, ld_kv = _rows2d(kv, "kv", 576, torch.bfloat16)
        kv_dtype, count, ld_cache = _kv_pool(kv_cache, kv_dtype)
        if n != rows:
            raise ValueError("kv must have %d rows" % rows)
    else:
        kv_dtype = IC_BF16
    if k is not None:
        n, ld_k = _rows2d(k, "k", 128, torch.bfloat16)
        if k_cache.dtype == torch.uint8:
            k_dt = IC_E4M3
        elif k_cache.dtype != torch.bfloat16:
            raise ValueError("k_cache must be bf16 or uint8")
        key_slots, ld = _pool(k_cache, "k_cache", k_cache.dtype)
        if n != rows or ld != 128 or k_cache.size(-1) != 128:
            raise ValueError("k must have %d rows, k_cache dense rows of 128" % rows)
        if count is not None and key_slots != count:
            raise ValueError("kv_cache and k_cache differ in their number of slots")
        count = key_slots
        if k_dt == IC_E4M3 and (k_scale is None or k_scale.dtype != torch.float32 or
                                k_scale.numel() != count or not k_scale.is_contiguous()):
            raise ValueError("an e4m3 key cache needs k_scale, fp32, one per slot")
    if rows == 0:
        return
    flags = (IC_ROPE_KV_HALVES if kv_halves else 0) | (IC_ROPE_K_HALVES if k_halves else 0)
    _launch(dev, stream, lib().ic_cache_append,
            rows, slots.data_ptr(), _ptr(pos), _ptr(rope), rope_rows, _ptr(kv), ld_kv,
            _ptr(kv_cache), ld_cache, kv_dtype, _ptr(k), ld_k, _ptr(k_cache), k_scale.data_ptr() if
            k_dt == IC_E4M3 else None, k_dt, count, flags)


def _paging(block_table, seq_lens, page_size, num_pages) -> ic_paging:
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [batch, max_pages]")
    batch, cols = block_table.shape
    ld = cols
    if not block_table.is_contiguous():
        if cols > 1 and block_table.stride(1) != 1:
            raise ValueError("block_table must have contiguous rows")
        if batch > 1:
            ld = block_table.stride(0)
    if seq_lens.dtype != torch.int32 or seq_lens.dim() != 1 or seq_lens.numel() != batch or \
            not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be int32 [batch], contiguous")
    return ic_paging(block_table.data_ptr(), ld, cols, seq_lens.data_ptr(), page_size, num_pages)


def make_paging(block_table, seq_lens, page_size: int, num_pages: int) -> ic_paging:
    """ic_paging over block_table [batch, max_pages] int32 and seq_lens [batch] int32, device
    tensors, which the result keeps alive."""
    pg = _paging(block_table, seq_lens, page_size, num_pages)
    _one_device(block_table, seq_lens)
    pg.tensors = (block_table, seq_lens)
    return pg


def _pages(rows, page_size, name):
    if page_size < 1 or rows % page_size:
        raise ValueError("%s must hold whole pages of %d rows" % (name, page_size))
    return rows // page_size


def ic_indexer_scores_paged(q, k_cache, w, block_table, seq_lens, *, page_size: int, scores=None,
                            q_scale=None, k_scale=None, stream=None):
    """Indexer scores [B, L] of one query per sequence (at its last token) over paged keys:
    q [B, 64, 128] or [B, 1, 64, 128], w [B(, 1), 64], k_cache [slots, 128] or [pages, page_size,
    128] (bf16, or uint8 e4m3 codes with q_scale [B(, 1), 64] and k_scale, one per slot).
    Writes columns s < seq_lens[b] of `scores` (new: [B, max_pages * page_size]) only."""
    dt = q.dtype
    if dt != torch.bfloat16 and dt != torch.uint8:
        raise ValueError("q must be bf16 or uint8 (e4m3 codes)")
    slots, ld = _pool(k_cache, "k_cache", dt)
    B, cols = block_table.shape
    H, d = q.shape[-2:]
    if d != k_cache.shape[-1] or ld != d:
        raise ValueError("q and k_cache must have dense rows of one length")
    BH = B * H
    if q.numel() != BH * d or w.dtype != torch.float32 or w.numel() != BH:
        raise ValueError("q must be [B, H, D] and w fp32 [B, H] with B = %d sequences" % B)
    _contig(q, w)
    fp8 = dt == torch.uint8
    if fp8:
        if q_scale is None or k_scale is None or q_scale.dtype != torch.float32 or \
                k_scale.dtype != torch.float32 or q_scale.numel() != BH or \
                k_scale.numel() != slots:
            raise ValueError("e4m3 keys need fp32 q_scale [B, H] and k_scale [slots]")
        _contig(q_scale, k_scale)
    dev = _one_device(q, k_cache, w, block_table, seq_lens, scores, q_scale, k_scale)
    pg = _paging(block_table, seq_lens, page_size, _pages(slots, page_size, "k_cache"))
    most = cols * page_size
    if scores is None:
        scores = _new((B, most), torch.float32, dev, stream)
    if scores.dtype != torch.float32 or scores.dim() != 2:
        raise ValueError("scores must be fp32 [%d, L]" % B)
    rows, width = scores.shape
    if rows != B:
        raise ValueError("scores must be fp32 [%d, L]" % B)
    ld = width
    if not scores.is_contiguous():
        if width > 1 and scores.stride(1) != 1:
            raise ValueError("scores must have contiguous rows")
        if B > 1:
            ld = scores.stride(0)
    _launch(dev, stream, lib().ic_indexer_scores_paged,
            q.data_ptr(), q_scale.data_ptr() if fp8 else None, k_cache.data_ptr(),
            k_scale.data_ptr() if fp8 else None, w.data_ptr(), IC_E4M3 if fp8 else IC_BF16, B, H,
            d, ctypes.byref(pg), width if width < most else most, scores.data_ptr(), ld)
    return scores


def ic_sparse_attn_paged(q, kv_cache, idx, block_table, seq_lens, scale: float, *, page_size: int,
                         kv_dtype=None, out=None, lse=None, workspace=None, stream=None):
    """Absorbed-MLA sparse attention over a paged latent cache: q [B, R, 16, 576] bf16, idx
    [B, R, k] int32 token numbers of each query's own sequence (entries outside it are
    skipped), kv_cache [slots, w] or [pages, page_size, w] of kv_dtype (IC_BF16; uint8 rows:
    IC_E4M3 or IC_MXF4).  workspace: ic_attn_workspace_size bytes let few queries be split."""
    if q.dtype != torch.bfloat16 or q.dim() != 4 or idx.dtype != torch.int32 or idx.dim() != 3:
        raise ValueError("q must be bf16 [B, R, H, D] and idx int32 [B, R, k]")
    B, R, H, dk = q.shape
    ib, ir, k = idx.shape
    if ib != B or ir != R or block_table.shape[0] != B:
        raise ValueError("q, idx and block_table must have one batch and one number of rows")
    _contig(q, idx, out, lse)
    kv_dtype, slots, ld = _kv_pool(kv_cache, kv_dtype)
    dev = _one_device(q, kv_cache, idx, block_table, seq_lens, out, lse, workspace)
    pg = _paging(block_table, seq_lens, page_size, _pages(slots, page_size, "kv_cache"))
    if out is None:
        out = _new((B, R, H, 512), torch.bfloat16, dev, stream)
    elif out.dtype != torch.bfloat16 or out.shape != (B, R, H, 512):
        raise ValueError("out must be bf16 %s" % ((B, R, H, 512),))
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (B, R, H)):
        raise ValueError("lse must be fp32 %s" % ((B, R, H),))
    ws, ws_bytes = (None, 0) if workspace is None else (
        workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if B and R == 0:
        return out
    _launch(dev, stream, lib().ic_sparse_attn_paged,
            q.data_ptr(), kv_cache.data_ptr(), ld, ctypes.byref(pg), idx.data_ptr(), kv_dtype, B,
            R, H, dk, 512, k, scale, out.data_ptr(), _ptr(lse), ws, ws_bytes)
    return out


_CODES = {IC_BF16: (torch.bfloat16,), IC_E4M3: (torch.uint8, torch.float8_e4m3fn),
          IC_MXF4: (torch.uint8,)}
_F32 = (torch.float32,)


def _holds(t, name, dtypes, count):
    """Refuses a tensor that is not contiguous, of none of the types or of fewer elements."""
    if t.dtype not in dtypes or not t.is_contiguous() or t.numel() < count:
        raise ValueError("%s must be contiguous %s of at least %d elements (got %s %s)" % (
            name, " or ".join(str(d) for d in dtypes), count, t.dtype, tuple(t.shape)))


def _check_step_paged(pattern, desc, paging, layers, t_cache, workspace) -> int:
    """The device of a paged decode step's tensors.  Refuses tensors on several devices, and
    those that hold less than desc and paging name, of another type, or with gaps.  Sizes and
    formats that no tensor could fit, and missing tensors, are left to the library."""
    B, rows = desc.batch, paging.num_pages * paging.page_size
    used = list(getattr(paging, "tensors", ()))
    if used and used[0].shape[0] < B:
        raise ValueError("desc.batch is %d, the block table has %d rows" % (B, used[0].shape[0]))
    if t_cache is not None:
        _holds(t_cache, "t_cache", (torch.int32,), B * desc.k)
        used.append(t_cache)
    if workspace is not None:
        _contig(workspace)
        used.append(workspace)
    heads = B * desc.heads
    fields = {"q": ((torch.bfloat16,), heads * desc.dk), "out": ((torch.bfloat16,), heads * desc.dv),
              "lse": (_F32, heads)}
    codes = _CODES.get(desc.idx_dtype)
    scores = {"q_idx": (codes, B * desc.H * desc.D), "k_idx": (codes, rows * desc.D),
              "w": (_F32, B * desc.H)}
    if desc.idx_dtype == IC_E4M3:
        scores.update(q_scale=(_F32, B * desc.H), k_scale=(_F32, rows))
    kv_codes = _CODES.get(desc.attn_dtype)
    kinds = [c for c in pattern if c in "FS"]
    for l, d in enumerate(layers):
        want = {**fields, **scores} if kinds[l:l + 1] == ["F"] else fields
        for f, (dtypes, count) in want.items():
            t = d.get(f)
            if t is not None:
                if dtypes is not None:
                    _holds(t, "layer %d: %s" % (l, f), dtypes, count)
                used.append(t)
        t = d.get("kv")
        if t is not None:
            if kv_codes is not None:
                name, width = "layer %d: kv" % l, _KV_ROW[desc.attn_dtype] // t.element_size()
                if t.is_contiguous():
                    _holds(t, name, kv_codes, (rows - 1) * desc.ld_kv + width)
                else:
                    if t.dtype not in kv_codes or t.shape[-1] < width:
                        raise ValueError("%s rows must be %s of at least %d elements" % (
                            name, kv_codes[0], width))
                    n, ld = _rows2d(t, name, t.shape[-1], t.dtype)
                    if n < rows or ld != desc.ld_kv:
                        raise ValueError("%s must hold %d rows, %d elements apart (got %d, %d)" % (
                            name, rows, desc.ld_kv, n, ld))
            used.append(t)
    return _one_device(*used) if used else torch.cuda.current_device()


def ic_decode_step_paged(pattern: str, desc: ic_stack_desc, paging: ic_paging, layers: list[dict],
                         t_cache, workspace, stream=None):
    """Decode step over paged caches (make_paging; desc.decode = 1, desc.L bounds the lengths):
    layers hold the pools as k_idx, k_scale and kv.  Runs on the tensors' device; tensors that
    hold less than desc and paging name are refused."""
    dev = _check_step_paged(pattern, desc, paging, layers, t_cache, workspace)
    arr = _layers(layers)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _launch(dev, stream, lib().ic_decode_step_paged, pattern.encode(), ctypes.byref(desc),
            ctypes.byref(paging), arr, len(layers), _ptr(t_cache), _ptr(workspace), ws_bytes)
