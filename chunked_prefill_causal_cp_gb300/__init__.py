"""Python binding of libcp.so, the GB300 chunked-prefill causal attention library.

Argument marshalling only: each function takes torch tensors (device memory
allocated by the caller), passes their pointers to the C entry point of the
same name declared in ``include/cp_api.h``, and raises ``CPError`` on a
non-zero status.  Every step of the computation runs in the library's CUDA
kernels; there is no fallback of any kind.  If the library has not been
built, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcp.so")

CP_OK = 0
CP_ERR_INVALID_ARG = -1
CP_ERR_UNSUPPORTED = -2
CP_ERR_CAPACITY = -3
CP_ERR_CUDA = -4
CP_ERR_WORKSPACE = -5
CP_DEV_BOUNDS = 1
CP_DEV_TIMEOUT = 2

CP_F32, CP_BF16, CP_F16 = 0, 1, 2
CP_CACHE_CONTIG, CP_CACHE_ROLLING, CP_CACHE_PAGED = 0, 1, 2
CP_TREE_MAX = 128

DTYPE_CODE = {torch.float32: CP_F32, torch.bfloat16: CP_BF16, torch.float16: CP_F16}


class LayerDesc(ctypes.Structure):
    """Mirror of ``cp_layer_desc``."""

    _fields_ = [
        ("dtype", c_int32), ("batch", c_int32), ("num_q_heads", c_int32),
        ("num_kv_heads", c_int32), ("head_dim", c_int32), ("kind", c_int32),
        ("capacity", c_int32), ("page_size", c_int32), ("num_pages", c_int32),
        ("max_blocks", c_int32), ("scale", c_float),
    ]


class SchedEntry(ctypes.Structure):
    """Mirror of ``cp_sched_entry``."""

    _fields_ = [("step", c_int32), ("seq", c_int32), ("start", c_int32), ("rows", c_int32)]


class QKPrep(ctypes.Structure):
    """Mirror of ``cp_qk_prep``."""

    _fields_ = [("rot_dim", c_int32), ("interleaved", c_int32), ("eps", c_float)]


class Q4Cache(ctypes.Structure):
    """Mirror of ``cp_q4_cache``; made by :func:`q4_cache`, it keeps its tensors alive."""

    _fields_ = [("k_codes", c_void_p), ("v_codes", c_void_p), ("k_params", c_void_p), ("v_params", c_void_p)]


class LatentDesc(ctypes.Structure):
    """Mirror of ``cp_latent_desc``."""

    _fields_ = [
        ("dtype", c_int32), ("batch", c_int32), ("num_heads", c_int32), ("latent_dim", c_int32), ("rope_dim", c_int32),
        ("nope_dim", c_int32), ("v_dim", c_int32), ("kind", c_int32), ("capacity", c_int32), ("page_size", c_int32),
        ("num_pages", c_int32), ("max_blocks", c_int32), ("scale", c_float),
    ]


class CPError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {cp_status_string(status)} ({status})")
        self.status = status


_lib = None


def lib():
    """The loaded libcp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P = c_void_p
        L.cp_kv_append.argtypes = [POINTER(LayerDesc), P, P, c_int32, P, P, P, P, c_int32, P, P]
        L.cp_pad_chunk.argtypes = [POINTER(LayerDesc), P, P, P, c_int32, c_int32, P]
        L.cp_prefill_chunk_attn.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, c_int32, c_int32,
                                            c_int32, P, P, c_size_t, c_int32, P, P]
        L.cp_prefill_chunk.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, P, P, c_int32, c_int32,
                                       c_int32, P, P, c_size_t, P, P]
        L.cp_mixed_step.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, P, P, c_int32, c_int32,
                                    c_int32, P, P, c_size_t, P, P]
        L.cp_mixed_step_overlap.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, P, P, c_int32, c_int32,
                                            c_int32, P, P, c_size_t, P, P, P, P, P]
        L.cp_prefill_varlen.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, P, c_int32, c_int32, c_int32, P,
                                        P, c_size_t, P, P]
        L.cp_prefill_varlen_overlap.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, P, c_int32, c_int32,
                                                c_int32, P, P, c_size_t, P, P, P, P, P]
        L.cp_mixed_step_noalloc.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, P, P, c_int32, c_int32,
                                            c_int32, P, P, P]
        L.cp_mixed_step_noalloc.restype = c_int32
        L.cp_noalloc_scratch_bytes.argtypes = []
        L.cp_noalloc_scratch_bytes.restype = c_size_t
        L.cp_workspace_size.argtypes = [POINTER(LayerDesc), c_int32, c_int32, c_int32]
        L.cp_workspace_size.restype = c_size_t
        L.cp_chunk_plan.argtypes = [c_int32, c_int32, POINTER(c_int32), c_int32]
        L.cp_query_ladder.argtypes = [c_int32, POINTER(c_int32)]
        L.cp_query_width.argtypes = [c_int32, c_int32]
        L.cp_aligned_length.argtypes = [c_int32, c_int32]
        L.cp_rolling_mask.argtypes = [c_int32, c_int32, c_int32, c_int32, POINTER(c_float)]
        L.cp_schedule.argtypes = [c_int32, c_int32, POINTER(c_int32), c_int32, POINTER(SchedEntry), c_int32]
        L.cp_status_string.argtypes = [c_int32]
        L.cp_selftest_bounded_wait.argtypes = [P, P, P]
        L.cp_abi_version.argtypes = []
        I, L64 = c_int32, c_int64
        L.cp_qk_norm_rope.argtypes = [POINTER(LayerDesc), POINTER(QKPrep), P, L64, P, L64, P, P, P, P, P, P, I, I, P,
                                      P, P]
        L.cp_qk_norm_rope_append.argtypes = [POINTER(LayerDesc), POINTER(QKPrep), P, L64, P, L64, P, L64, P, P, P, P,
                                             P, I, I, P, P, P, P, P, I, P, P]
        L.cp_kv_append_q4.argtypes = [POINTER(LayerDesc), P, P, P, I, I, POINTER(Q4Cache), P, P, I, P, P]
        L.cp_kv_read_q4.argtypes = [POINTER(LayerDesc), POINTER(Q4Cache), P, P, P, I, I, I, P, P, P, P]
        L.cp_chunk_attn_q4.argtypes = [POINTER(LayerDesc), P, POINTER(Q4Cache), P, P, P, I, I, I, P, P, c_size_t, I,
                                       P, P]
        L.cp_mixed_step_q4.argtypes = [POINTER(LayerDesc), P, P, P, POINTER(Q4Cache), P, P, P, I, I, I, P, P,
                                       c_size_t, I, P, P]
        L.cp_workspace_size_q4.argtypes = [POINTER(LayerDesc), I, I, I]
        L.cp_workspace_size_q4.restype = c_size_t
        LD = POINTER(LatentDesc)
        L.cp_latent_append.argtypes = [LD, POINTER(QKPrep), P, L64, P, L64, P, P, P, P, L64, L64, P, L64, L64, P, I, I,
                                       P, P, P, I, P, P]
        L.cp_latent_attn.argtypes = [LD, P, P, P, P, P, P, I, I, I, P, P, c_size_t, I, P, P]
        L.cp_workspace_size_latent.argtypes = [LD, I, I, I]
        L.cp_workspace_size_latent.restype = c_size_t
        L.cp_latent_chunk_attn.argtypes = [LD, P, P, L64, L64, P, L64, P, L64, L64, P, P, I, I, I, P, P, P]
        L.cp_tree_attn.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, P, I, I, I, P, P, c_size_t, P, P]
        L.cp_workspace_size_tree.argtypes = [POINTER(LayerDesc), I, I, I]
        L.cp_workspace_size_tree.restype = c_size_t
        L.cp_tree_commit.argtypes = [POINTER(LayerDesc), P, P, P, P, P, P, I, I, I, I, P, P]
        L.cp_latent_tree_commit.argtypes = [LD, P, P, P, P, P, I, I, I, I, P, P]
        L.cp_status_string.restype = ctypes.c_char_p
        for name in ("cp_kv_append", "cp_pad_chunk", "cp_prefill_chunk_attn", "cp_prefill_chunk",
                     "cp_mixed_step", "cp_mixed_step_overlap", "cp_prefill_varlen", "cp_prefill_varlen_overlap",
                     "cp_chunk_plan",
                     "cp_query_ladder", "cp_query_width", "cp_aligned_length", "cp_rolling_mask",
                     "cp_schedule", "cp_abi_version", "cp_selftest_bounded_wait",
                     "cp_qk_norm_rope", "cp_qk_norm_rope_append", "cp_kv_append_q4", "cp_kv_read_q4",
                     "cp_chunk_attn_q4", "cp_mixed_step_q4", "cp_latent_append", "cp_latent_attn",
                     "cp_latent_chunk_attn", "cp_tree_attn", "cp_tree_commit", "cp_latent_tree_commit"):
            getattr(L, name).restype = c_int32
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, *tensors):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            return torch.cuda.current_stream(t.device).cuda_stream
    return None


def _check(status: int, where: str):
    if status != CP_OK:
        raise CPError(status, where)


def layer_desc(dtype, batch, num_q_heads, num_kv_heads, head_dim, kind=CP_CACHE_CONTIG,
               capacity=0, page_size=0, num_pages=0, max_blocks=0, scale=0.0) -> LayerDesc:
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return LayerDesc(code, batch, num_q_heads, num_kv_heads, head_dim, kind, capacity, page_size,
                     num_pages, max_blocks, scale)


def cp_kv_append(desc, k_new, v_new, rows, k_cache, v_cache, seqlens_k, max_past,
                 block_table=None, dev_status=None, stream=None):
    s = lib().cp_kv_append(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), rows, _ptr(k_cache),
                           _ptr(v_cache), _ptr(seqlens_k), _ptr(block_table), max_past,
                           _ptr(dev_status), _stream(stream, k_new))
    _check(s, "cp_kv_append")


def cp_pad_chunk(desc, q, k_new, v_new, real_rows, rows_padded, stream=None):
    s = lib().cp_pad_chunk(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), real_rows, rows_padded,
                           _stream(stream, q, k_new, v_new))
    _check(s, "cp_pad_chunk")


def cp_prefill_chunk_attn(desc, q, k_cache, v_cache, seqlens_k, rows_padded, real_rows, max_past,
                          out, workspace=None, commit=True, block_table=None, left_pad=None,
                          dev_status=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    s = lib().cp_prefill_chunk_attn(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(seqlens_k), _ptr(block_table), _ptr(left_pad), rows_padded,
                                    real_rows, max_past, _ptr(out), _ptr(workspace), ws_bytes,
                                    1 if commit else 0, _ptr(dev_status), _stream(stream, q))
    _check(s, "cp_prefill_chunk_attn")


def cp_prefill_chunk(desc, q, k_new, v_new, k_cache, v_cache, seqlens_k, rows_padded, real_rows, max_past,
                     out, workspace, block_table=None, left_pad=None, dev_status=None, stream=None):
    """Append, attention and commit of one chunk in one call (see include/cp_api.h)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    s = lib().cp_prefill_chunk(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                               _ptr(v_cache), _ptr(seqlens_k), _ptr(block_table), _ptr(left_pad), rows_padded,
                               real_rows, max_past, _ptr(out), _ptr(workspace), ws_bytes, _ptr(dev_status),
                               _stream(stream, q))
    _check(s, "cp_prefill_chunk")


def cp_mixed_step(desc, q, k_new, v_new, k_pages, v_pages, block_table, cu_rows, past_len,
                  num_seqs, total_rows, max_ctx, out, workspace, dev_status=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    s = lib().cp_mixed_step(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages),
                            _ptr(v_pages), _ptr(block_table), _ptr(cu_rows), _ptr(past_len), num_seqs,
                            total_rows, max_ctx, _ptr(out), _ptr(workspace), ws_bytes,
                            _ptr(dev_status), _stream(stream, q))
    _check(s, "cp_mixed_step")


def _side_handles(side_stream, fork_event, join_event):
    """Raw handles of a side stream and two events (torch objects or raw handles)."""
    side = side_stream if isinstance(side_stream, int) else side_stream.cuda_stream
    evs = []
    for ev in (fork_event, join_event):
        if isinstance(ev, int):
            evs.append(ev)
            continue
        if not ev.cuda_event:  # torch creates the event on its first record
            ev.record(side_stream if not isinstance(side_stream, int) else None)
        evs.append(ev.cuda_event)
    return side, evs


def cp_mixed_step_overlap(desc, q, k_new, v_new, k_pages, v_pages, block_table, cu_rows, past_len,
                          num_seqs, total_rows, max_ctx, out, workspace, side_stream, fork_event, join_event,
                          dev_status=None, stream=None):
    """cp_mixed_step with the split-KV kernels on `side_stream` beside the
    tensor-core kernel (see include/cp_api.h).  `side_stream` is a
    torch.cuda.Stream (or a raw handle); the events are torch.cuda.Event
    objects (or raw handles)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    side, evs = _side_handles(side_stream, fork_event, join_event)
    s = lib().cp_mixed_step_overlap(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages),
                                    _ptr(v_pages), _ptr(block_table), _ptr(cu_rows), _ptr(past_len), num_seqs,
                                    total_rows, max_ctx, _ptr(out), _ptr(workspace), ws_bytes,
                                    _ptr(dev_status), _stream(stream, q), side, evs[0], evs[1])
    _check(s, "cp_mixed_step_overlap")


def cp_prefill_varlen(desc, q, k_new, v_new, k_cache, v_cache, cu_rows, seqlens_k, num_seqs, total_rows, max_ctx,
                      out, workspace, dev_status=None, stream=None):
    """Several sequences with ragged rows over a contiguous cache in one call (see include/cp_api.h)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    s = lib().cp_prefill_varlen(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                _ptr(v_cache), _ptr(cu_rows), _ptr(seqlens_k), num_seqs, total_rows, max_ctx,
                                _ptr(out), _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream, q))
    _check(s, "cp_prefill_varlen")


def cp_prefill_varlen_overlap(desc, q, k_new, v_new, k_cache, v_cache, cu_rows, seqlens_k, num_seqs, total_rows,
                              max_ctx, out, workspace, side_stream, fork_event, join_event, dev_status=None,
                              stream=None):
    """cp_prefill_varlen with the one-row sequences' split-KV kernels on
    `side_stream` (see include/cp_api.h); handles as in cp_mixed_step_overlap."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    side, evs = _side_handles(side_stream, fork_event, join_event)
    s = lib().cp_prefill_varlen_overlap(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                        _ptr(v_cache), _ptr(cu_rows), _ptr(seqlens_k), num_seqs, total_rows,
                                        max_ctx, _ptr(out), _ptr(workspace), ws_bytes, _ptr(dev_status),
                                        _stream(stream, q), side, evs[0], evs[1])
    _check(s, "cp_prefill_varlen_overlap")


def cp_mixed_step_noalloc(desc, q, k_new, v_new, k_pages, v_pages, block_table, cu_rows, past_len,
                          num_seqs, total_rows, max_ctx, out, dev_status=None, stream=None):
    """cp_mixed_step without a workspace: the split-KV scratch is a fixed array
    inside the library (see include/cp_api.h for its limit and sharing rules)."""
    s = lib().cp_mixed_step_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages),
                                    _ptr(v_pages), _ptr(block_table), _ptr(cu_rows), _ptr(past_len),
                                    num_seqs, total_rows, max_ctx, _ptr(out), _ptr(dev_status),
                                    _stream(stream, q))
    _check(s, "cp_mixed_step_noalloc")


# ---- queries and keys before attention, and the cache held in 4 bits.  Beyond
# marshalling, these refuse (CPError, CP_ERR_INVALID_ARG) a tensor whose type,
# device or strides are not what the call takes, instead of reading it wrongly.

def _refuse(where):
    raise CPError(CP_ERR_INVALID_ARG, where)


def _device(where, *tensors):
    """Index of the first tensor's device, which has to be the current one: the library launches there.  The current one
    when all are raw handles."""
    for t in tensors:
        if isinstance(t, torch.Tensor):
            dev = t.get_device()
            if dev < 0 or dev != torch._C._cuda_getDevice():
                _refuse(where)
            return dev
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else 0


def _on(dev, stream):
    """The given stream, or the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _arg(where, t, dtype, numel, dev):
    """Pointer of a dense tensor of `dtype` on `dev` with at least `numel` elements.  None (which the library
    refuses where it may not be) and raw handles pass."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    _refuse(where)


_LAYER_DTYPE = {code: dtype for dtype, code in DTYPE_CODE.items()}


def _workspace(where, t, dev):
    """Pointer and bytes of a workspace."""
    if t is None or isinstance(t, int):
        return t, 0
    if t.get_device() != dev or not t.is_contiguous():
        _refuse(where)
    return t.data_ptr(), t.numel() * t.element_size()


def _rows_arg(where, t, desc, heads, total_rows, dev):
    """(pointer, row stride in elements) of rows [..., heads, D]: a head row is dense, and one stride leads from
    each row to the next.  None and raw handles pass as they are (dense)."""
    if t is None or isinstance(t, int):
        return t, 0
    d, n, shape = desc.head_dim, t.numel(), t.shape
    if (t.dtype is not _LAYER_DTYPE.get(desc.dtype) or t.get_device() != dev or len(shape) < 2 or shape[-1] != d
            or shape[-2] != heads or n != total_rows * heads * d):
        _refuse(where)
    if n == 0 or t.is_contiguous():
        return t.data_ptr(), 0
    if t.stride(-1) != 1 or (heads > 1 and t.stride(-2) != d):
        _refuse(where)
    stride = size = None  # of the rows so far, from the last dimension of rows
    for n, st in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n == 1:
            continue
        if stride is None:
            stride, size = st, n
        elif st == stride * size:
            size *= n
        else:
            _refuse(where)
    if stride is not None and stride < 1:  # an expanded tensor's rows: 0 would read as dense
        _refuse(where)
    return t.data_ptr(), stride or 0


def qk_prep(rot_dim, interleaved=False, eps=1e-6) -> QKPrep:
    return QKPrep(rot_dim, 1 if interleaved else 0, eps)


def q4_cache(k_codes, v_codes, k_params, v_params) -> Q4Cache:
    """The arrays of a 4-bit cache, on one device: uint8 codes [..., D / 2] and params [..., D / 32, 2] of the layer's
    type."""
    for c, p in ((k_codes, k_params), (v_codes, v_params)):
        if (c.dtype != torch.uint8 or p.dtype not in (torch.bfloat16, torch.float16) or not c.is_contiguous()
                or not p.is_contiguous() or not c.is_cuda or not p.is_cuda or p.dim() < 2 or p.shape[-1] != 2
                or tuple(c.shape) != (*p.shape[:-2], p.shape[-2] * 16)):
            _refuse("q4_cache")
    if (k_codes.shape != v_codes.shape or k_params.dtype != v_params.dtype
            or len({x.get_device() for x in (k_codes, v_codes, k_params, v_params)}) != 1):
        _refuse("q4_cache")
    c = Q4Cache(k_codes.data_ptr(), v_codes.data_ptr(), k_params.data_ptr(), v_params.data_ptr())
    c.tensors = (k_codes, v_codes, k_params, v_params)
    return c


def _q4_arg(where, desc, cache, dev):
    """The cache, with arrays as large as desc says."""
    tensors = getattr(cache, "tensors", None)
    if tensors is not None:
        slots = desc.num_pages * desc.page_size if desc.kind == CP_CACHE_PAGED else desc.batch * desc.capacity
        codes, params = tensors[0], tensors[2]
        if (params.dtype is not _LAYER_DTYPE.get(desc.dtype) or codes.get_device() != dev
                or codes.numel() < slots * desc.num_kv_heads * (desc.head_dim // 2)):
            _refuse(where)
    return ctypes.byref(cache)


def _seq_args(where, desc, lens, cu_rows, block_table, num_seqs, dev):
    return (_arg(where, lens, torch.int32, num_seqs, dev), _arg(where, cu_rows, torch.int32, num_seqs + 1, dev),
            _arg(where, block_table, torch.int32, num_seqs * desc.max_blocks, dev))


def cp_qk_norm_rope(desc, prep, q, k, q_out, k_out, num_seqs, total_rows, q_weight=None, k_weight=None, inv_freq=None,
                    positions=None, seqlens_k=None, cu_rows=None, stream=None):
    """Norm of every query and key head and rotary position, one pass (see include/cp_api.h).  q and k may be
    slices of a projection's rows."""
    w, dt, d, i32 = "cp_qk_norm_rope", _LAYER_DTYPE.get(desc.dtype), desc.head_dim, torch.int32
    hq, hkv = desc.num_q_heads, desc.num_kv_heads
    dev = _device(w, q, k)
    pq, sq = _rows_arg(w, q, desc, hq, total_rows, dev)
    pk, sk = _rows_arg(w, k, desc, hkv, total_rows, dev)
    s = lib().cp_qk_norm_rope(
        ctypes.byref(desc), ctypes.byref(prep), pq, sq, pk, sk, _arg(w, q_weight, dt, d, dev),
        _arg(w, k_weight, dt, d, dev), _arg(w, inv_freq, torch.float32, prep.rot_dim // 2, dev),
        _arg(w, positions, i32, total_rows, dev), _arg(w, seqlens_k, i32, num_seqs, dev),
        _arg(w, cu_rows, i32, num_seqs + 1, dev), num_seqs, total_rows, _arg(w, q_out, dt, total_rows * hq * d, dev),
        _arg(w, k_out, dt, total_rows * hkv * d, dev), _on(dev, stream))
    _check(s, w)


def cp_qk_norm_rope_append(desc, prep, q, k_new, v_new, q_out, k_cache, v_cache, seqlens_k, num_seqs, total_rows,
                           max_ctx, q_weight=None, k_weight=None, inv_freq=None, positions=None, cu_rows=None,
                           block_table=None, dev_status=None, stream=None):
    """cp_qk_norm_rope with the keys and values into their cache slots (see include/cp_api.h)."""
    w, dt, d, i32 = "cp_qk_norm_rope_append", _LAYER_DTYPE.get(desc.dtype), desc.head_dim, torch.int32
    hq, hkv = desc.num_q_heads, desc.num_kv_heads
    dev = _device(w, q, k_new, v_new)
    pq, sq = _rows_arg(w, q, desc, hq, total_rows, dev)
    pk, sk = _rows_arg(w, k_new, desc, hkv, total_rows, dev)
    pv, sv = _rows_arg(w, v_new, desc, hkv, total_rows, dev)
    size = (desc.num_pages * desc.page_size if desc.kind == CP_CACHE_PAGED else desc.batch * desc.capacity) * hkv * d
    lens, cu, table = _seq_args(w, desc, seqlens_k, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_qk_norm_rope_append(
        ctypes.byref(desc), ctypes.byref(prep), pq, sq, pk, sk, pv, sv, _arg(w, q_weight, dt, d, dev),
        _arg(w, k_weight, dt, d, dev), _arg(w, inv_freq, torch.float32, prep.rot_dim // 2, dev),
        _arg(w, positions, i32, total_rows, dev), cu, num_seqs, total_rows, _arg(w, q_out, dt, total_rows * hq * d, dev),
        _arg(w, k_cache, dt, size, dev), _arg(w, v_cache, dt, size, dev), lens, table, max_ctx,
        _arg(w, dev_status, i32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_kv_append_q4(desc, k_new, v_new, cache, seqlens_k, num_seqs, total_rows, max_ctx, cu_rows=None,
                    block_table=None, dev_status=None, stream=None):
    """Rows into a 4-bit cache (see include/cp_api.h)."""
    w, dt, n = "cp_kv_append_q4", _LAYER_DTYPE.get(desc.dtype), total_rows * desc.num_kv_heads * desc.head_dim
    dev = _device(w, k_new, v_new)
    lens, cu, table = _seq_args(w, desc, seqlens_k, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_kv_append_q4(ctypes.byref(desc), _arg(w, k_new, dt, n, dev), _arg(w, v_new, dt, n, dev), cu, num_seqs,
                              total_rows, _q4_arg(w, desc, cache, dev), lens, table, max_ctx,
                              _arg(w, dev_status, torch.int32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_kv_read_q4(desc, cache, starts, num_seqs, total_rows, max_ctx, k_out, v_out, cu_rows=None, block_table=None,
                  dev_status=None, stream=None):
    """The values that rows of a 4-bit cache stand for (see include/cp_api.h)."""
    w, dt, n = "cp_kv_read_q4", _LAYER_DTYPE.get(desc.dtype), total_rows * desc.num_kv_heads * desc.head_dim
    dev = _device(w, starts)
    lens, cu, table = _seq_args(w, desc, starts, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_kv_read_q4(ctypes.byref(desc), _q4_arg(w, desc, cache, dev), lens, table, cu, num_seqs, total_rows,
                            max_ctx, _arg(w, k_out, dt, n, dev), _arg(w, v_out, dt, n, dev),
                            _arg(w, dev_status, torch.int32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_chunk_attn_q4(desc, q, cache, seqlens_k, num_seqs, total_rows, max_ctx, out, workspace, cu_rows=None,
                     block_table=None, commit=True, dev_status=None, stream=None):
    """Causal attention over a 4-bit cache (see include/cp_api.h)."""
    w, dt, n = "cp_chunk_attn_q4", _LAYER_DTYPE.get(desc.dtype), total_rows * desc.num_q_heads * desc.head_dim
    dev = _device(w, q, out)
    ws, ws_bytes = _workspace(w, workspace, dev)
    lens, cu, table = _seq_args(w, desc, seqlens_k, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_chunk_attn_q4(ctypes.byref(desc), _arg(w, q, dt, n, dev), _q4_arg(w, desc, cache, dev), lens, table,
                               cu, num_seqs, total_rows, max_ctx, _arg(w, out, dt, n, dev), ws, ws_bytes,
                               1 if commit else 0, _arg(w, dev_status, torch.int32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_mixed_step_q4(desc, q, k_new, v_new, cache, seqlens_k, num_seqs, total_rows, max_ctx, out, workspace,
                     cu_rows=None, block_table=None, commit=True, dev_status=None, stream=None):
    """Append, attention and advance of a step over a 4-bit cache in one call (see include/cp_api.h)."""
    w, dt, d = "cp_mixed_step_q4", _LAYER_DTYPE.get(desc.dtype), desc.head_dim
    nq, nk = total_rows * desc.num_q_heads * d, total_rows * desc.num_kv_heads * d
    dev = _device(w, q, out)
    ws, ws_bytes = _workspace(w, workspace, dev)
    lens, cu, table = _seq_args(w, desc, seqlens_k, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_mixed_step_q4(ctypes.byref(desc), _arg(w, q, dt, nq, dev), _arg(w, k_new, dt, nk, dev),
                               _arg(w, v_new, dt, nk, dev), _q4_arg(w, desc, cache, dev), table, cu, lens, num_seqs,
                               total_rows, max_ctx, _arg(w, out, dt, nq, dev), ws, ws_bytes, 1 if commit else 0,
                               _arg(w, dev_status, torch.int32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_workspace_size_q4(desc, total_rows, max_ctx, num_seqs) -> int:
    return int(lib().cp_workspace_size_q4(ctypes.byref(desc), total_rows, max_ctx, num_seqs))


# ---- latent caches and drafted trees; tensors are refused as in the calls above.

def latent_desc(dtype, batch, num_heads, latent_dim, rope_dim, nope_dim=128, v_dim=128, kind=CP_CACHE_CONTIG, capacity=0,
                page_size=0, num_pages=0, max_blocks=0, scale=0.0) -> LatentDesc:
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return LatentDesc(code, batch, num_heads, latent_dim, rope_dim, nope_dim, v_dim, kind, capacity, page_size, num_pages,
                      max_blocks, scale)


def _rows2_arg(where, t, dtype, rows, width, dev):
    """(pointer, row stride) of rows [rows, width] whose channels are dense and whose stride leads forward.  None and raw
    handles pass as they are (dense)."""
    if t is None or isinstance(t, int):
        return t, 0
    if t.dtype is dtype and t.get_device() == dev and t.shape == (rows, width):
        s0, s1 = t.stride()
        if rows < 2 or width < 1:  # a single row has any stride
            s0 = width
        if s0 >= width and (s1 == 1 or width < 2 or rows < 1):
            return t.data_ptr(), s0
    _refuse(where)


def _rows3_arg(where, t, dtype, rows, heads, width, dev):
    """(pointer, row stride, head stride) of [rows, heads, width], as _rows2_arg."""
    if t is None or isinstance(t, int):
        return t, 0, 0
    if t.dtype is dtype and t.get_device() == dev and t.shape == (rows, heads, width):
        s0, s1, s2 = t.stride()
        if heads < 2 or rows < 1 or width < 1:
            s1 = width
        if rows < 2 or width < 1:
            s0 = s1 * heads
        if s1 >= width and s0 >= s1 * heads and (s2 == 1 or width < 2 or rows < 1):
            return t.data_ptr(), s0, s1
    _refuse(where)


def _slots(desc):
    return desc.num_pages * desc.page_size if desc.kind == CP_CACHE_PAGED else desc.batch * desc.capacity


def cp_latent_append(desc, prep, latent, k_rope, cache, seqlens_k, num_seqs, total_rows, max_ctx, weight=None,
                     inv_freq=None, positions=None, q_rope=None, q_out=None, cu_rows=None, block_table=None,
                     dev_status=None, stream=None):
    """Norm of the latents [T, C], rotary position of the shared keys [T, R] and of the queries' parts [T, H, R], rows
    into a latent cache (see include/cp_api.h).  All of them may be slices of projections' rows, q_out [T, H, R] of a
    buffer of wider heads."""
    w, dt, c, r, i32 = "cp_latent_append", _LAYER_DTYPE.get(desc.dtype), desc.latent_dim, desc.rope_dim, torch.int32
    dev = _device(w, latent)
    pl, sl = _rows2_arg(w, latent, dt, total_rows, c, dev)
    pk, sk = _rows2_arg(w, k_rope, dt, total_rows, r, dev)
    pq, qr, qh = _rows3_arg(w, q_rope, dt, total_rows, desc.num_heads, r, dev)
    po, outr, outh = _rows3_arg(w, q_out, dt, total_rows, desc.num_heads, r, dev)
    lens, cu, table = _seq_args(w, desc, seqlens_k, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_latent_append(
        ctypes.byref(desc), ctypes.byref(prep), pl, sl, pk, sk, _arg(w, weight, dt, c, dev),
        _arg(w, inv_freq, torch.float32, prep.rot_dim // 2, dev), _arg(w, positions, i32, total_rows, dev), pq, qr, qh,
        po, outr, outh, cu, num_seqs, total_rows, _arg(w, cache, dt, _slots(desc) * (c + r), dev), lens, table, max_ctx,
        _arg(w, dev_status, i32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_latent_attn(desc, q, cache, seqlens_k, num_seqs, total_rows, max_ctx, out, workspace, parents=None, cu_rows=None,
                   block_table=None, commit=True, dev_status=None, stream=None):
    """Attention over a latent cache, absorbed form: rows that follow one another, or with `parents` (and commit=False)
    the nodes of drafted trees (see include/cp_api.h)."""
    w, dt, c, r, i32 = "cp_latent_attn", _LAYER_DTYPE.get(desc.dtype), desc.latent_dim, desc.rope_dim, torch.int32
    n = total_rows * desc.num_heads
    dev = _device(w, q, out)
    ws, ws_bytes = _workspace(w, workspace, dev)
    lens, cu, table = _seq_args(w, desc, seqlens_k, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_latent_attn(
        ctypes.byref(desc), _arg(w, q, dt, n * (c + r), dev), _arg(w, cache, dt, _slots(desc) * (c + r), dev), lens, table,
        _arg(w, parents, i32, total_rows, dev), cu, num_seqs, total_rows, max_ctx, _arg(w, out, dt, n * c, dev), ws,
        ws_bytes, 1 if commit else 0, _arg(w, dev_status, i32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_workspace_size_latent(desc, total_rows, max_ctx, num_seqs) -> int:
    return int(lib().cp_workspace_size_latent(ctypes.byref(desc), total_rows, max_ctx, num_seqs))


def cp_latent_chunk_attn(desc, q, k_nope, k_rope, v, out, num_seqs, total_rows, total_keys, cu_rows=None, cu_keys=None,
                         dev_status=None, stream=None):
    """Attention of prompt chunks over expanded keys [N, H, nope_dim], shared rotated keys [N, R] and values [N, H,
    v_dim], which may be slices of wider rows (see include/cp_api.h)."""
    w, dt, h = "cp_latent_chunk_attn", _LAYER_DTYPE.get(desc.dtype), desc.num_heads
    dn, r, dv, i32 = desc.nope_dim, desc.rope_dim, desc.v_dim, torch.int32
    dev = _device(w, q, out)
    pk, kr, kh = _rows3_arg(w, k_nope, dt, total_keys, h, dn, dev)
    pr, rr = _rows2_arg(w, k_rope, dt, total_keys, r, dev)
    pv, vr, vh = _rows3_arg(w, v, dt, total_keys, h, dv, dev)
    s = lib().cp_latent_chunk_attn(
        ctypes.byref(desc), _arg(w, q, dt, total_rows * h * (dn + r), dev), pk, kr, kh, pr, rr, pv, vr, vh,
        _arg(w, cu_rows, i32, num_seqs + 1, dev), _arg(w, cu_keys, i32, num_seqs + 1, dev), num_seqs, total_rows,
        total_keys, _arg(w, out, dt, total_rows * h * dv, dev), _arg(w, dev_status, i32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_tree_attn(desc, q, k_cache, v_cache, seqlens_k, parents, num_seqs, total_rows, max_ctx, out, workspace,
                 cu_rows=None, block_table=None, dev_status=None, stream=None):
    """Attention of a drafted tree's nodes over a K/V cache (see include/cp_api.h)."""
    w, dt, d, i32 = "cp_tree_attn", _LAYER_DTYPE.get(desc.dtype), desc.head_dim, torch.int32
    n, size = total_rows * desc.num_q_heads * d, _slots(desc) * desc.num_kv_heads * d
    dev = _device(w, q, out)
    ws, ws_bytes = _workspace(w, workspace, dev)
    lens, cu, table = _seq_args(w, desc, seqlens_k, cu_rows, block_table, num_seqs, dev)
    s = lib().cp_tree_attn(
        ctypes.byref(desc), _arg(w, q, dt, n, dev), _arg(w, k_cache, dt, size, dev), _arg(w, v_cache, dt, size, dev), lens,
        table, _arg(w, parents, i32, total_rows, dev), cu, num_seqs, total_rows, max_ctx, _arg(w, out, dt, n, dev), ws,
        ws_bytes, _arg(w, dev_status, i32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_workspace_size_tree(desc, total_rows, max_ctx, num_seqs) -> int:
    return int(lib().cp_workspace_size_tree(ctypes.byref(desc), total_rows, max_ctx, num_seqs))


def cp_tree_commit(desc, k_cache, v_cache, path, counts, seqlens_k, num_seqs, max_path, max_ctx, block_table=None,
                   commit=True, dev_status=None, stream=None):
    """The rows of each sequence's accepted path moved to their places in a K/V cache (see include/cp_api.h)."""
    w, dt, i32 = "cp_tree_commit", _LAYER_DTYPE.get(desc.dtype), torch.int32
    size = _slots(desc) * desc.num_kv_heads * desc.head_dim
    dev = _device(w, k_cache, v_cache)
    lens, _, table = _seq_args(w, desc, seqlens_k, None, block_table, num_seqs, dev)
    s = lib().cp_tree_commit(
        ctypes.byref(desc), _arg(w, k_cache, dt, size, dev), _arg(w, v_cache, dt, size, dev),
        _arg(w, path, i32, num_seqs * max_path, dev), _arg(w, counts, i32, num_seqs, dev), lens, table, num_seqs, max_path,
        max_ctx, 1 if commit else 0, _arg(w, dev_status, i32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_latent_tree_commit(desc, cache, path, counts, seqlens_k, num_seqs, max_path, max_ctx, block_table=None,
                          commit=True, dev_status=None, stream=None):
    """cp_tree_commit on a latent cache (see include/cp_api.h)."""
    w, dt, i32 = "cp_latent_tree_commit", _LAYER_DTYPE.get(desc.dtype), torch.int32
    dev = _device(w, cache)
    lens, _, table = _seq_args(w, desc, seqlens_k, None, block_table, num_seqs, dev)
    s = lib().cp_latent_tree_commit(
        ctypes.byref(desc), _arg(w, cache, dt, _slots(desc) * (desc.latent_dim + desc.rope_dim), dev),
        _arg(w, path, i32, num_seqs * max_path, dev), _arg(w, counts, i32, num_seqs, dev), lens, table, num_seqs, max_path,
        max_ctx, 1 if commit else 0, _arg(w, dev_status, i32, 1, dev), _on(dev, stream))
    _check(s, w)


def cp_noalloc_scratch_bytes() -> int:
    return int(lib().cp_noalloc_scratch_bytes())


def cp_workspace_size(desc, max_rows, max_ctx, num_seqs) -> int:
    return int(lib().cp_workspace_size(ctypes.byref(desc), max_rows, max_ctx, num_seqs))


def cp_chunk_plan(n_tokens, chunk):
    n = lib().cp_chunk_plan(n_tokens, chunk, None, 0)
    _check(min(n, 0), "cp_chunk_plan")
    buf = (c_int32 * max(n, 1))()
    lib().cp_chunk_plan(n_tokens, chunk, buf, n)
    return list(buf[:n])


def cp_query_ladder(chunk):
    buf = (c_int32 * 3)()
    n = lib().cp_query_ladder(chunk, buf)
    _check(min(n, 0), "cp_query_ladder")
    return list(buf[:n])


def cp_query_width(real_rows, chunk):
    w = lib().cp_query_width(real_rows, chunk)
    _check(min(w, 0), "cp_query_width")
    return w


def cp_aligned_length(n_real, c):
    v = lib().cp_aligned_length(n_real, c)
    _check(min(v, 0), "cp_aligned_length")
    return v


def cp_rolling_mask(c, C, chunk_idx, left_pad):
    buf = (c_float * (c * C))()
    _check(lib().cp_rolling_mask(c, C, chunk_idx, left_pad, buf), "cp_rolling_mask")
    return torch.frombuffer(bytearray(buf), dtype=torch.float32).reshape(c, C)


def cp_schedule(budget, n_running, prompt_lens):
    arr = (c_int32 * max(len(prompt_lens), 1))(*prompt_lens)
    n = lib().cp_schedule(budget, n_running, arr, len(prompt_lens), None, 0)
    _check(min(n, 0), "cp_schedule")
    buf = (SchedEntry * max(n, 1))()
    lib().cp_schedule(budget, n_running, arr, len(prompt_lens), buf, n)
    return [(e.step, e.seq, e.start, e.rows) for e in buf[:n]]


def cp_status_string(status) -> str:
    return lib().cp_status_string(status).decode()


def cp_abi_version() -> int:
    return lib().cp_abi_version()


def cp_selftest_bounded_wait(dev_status, dev_out, stream=None) -> int:
    return lib().cp_selftest_bounded_wait(_ptr(dev_status), _ptr(dev_out), _stream(stream, dev_out))
