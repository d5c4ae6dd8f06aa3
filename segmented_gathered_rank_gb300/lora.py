"""Thin ctypes binding of ``include/lora.h`` (argument marshalling only).

Every function has the name of the C entry point it calls.  Device arguments
are CUDA torch tensors (their data pointers are passed), host arrays for
``lora_pool_load`` are numpy arrays or CPU tensors, and ``stream`` defaults to
torch's current stream.  A non-zero status raises :class:`LoraError`.  All
arithmetic happens in the CUDA library; importing this module fails when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

from . import build as _build

LORA_OK = 0
LORA_ERR_ARG = -1
LORA_ERR_POOL_FULL = -2
LORA_ERR_RANK = -3
LORA_ERR_NOT_LOADED = -4
LORA_ERR_CUDA = -5
LORA_ERR_DEVICE_INDEX = -6
LORA_ERR_SHAPE = -7

LORA_F32 = 0
LORA_BF16 = 1

LORA_DEV_BAD_ADAPTER = 1
LORA_DEV_BAD_SEGMENTS = 2
LORA_DEV_WAIT_TIMEOUT = 4
LORA_DEV_BAD_SLOT = 8
LORA_DEV_BAD_POSITION = 16
LORA_DEV_BAD_LENGTH = 32
LORA_DEV_BAD_PAGE = 64

LORA_NOALLOC_SCRATCH_BYTES = 16 << 20
LORA_MAX_AXES = 4

LORA_TIER_GPU = 0
LORA_TIER_HOST = 1
LORA_TIER_DISK = 2

EXPORTS = ["lora_pool_create", "lora_pool_destroy", "lora_pool_load", "lora_pool_unload",
           "lora_pool_free_pages", "lora_sgmv_shrink", "lora_sgmv_expand", "lora_bgmv",
           "lora_layer_forward_workspace_size", "lora_layer_forward", "lora_get_error", "lora_strerror",
           "lora_launch_count", "lora_layer_forward_noalloc", "lora_tier_cache_create", "lora_tier_cache_destroy",
           "lora_tier_cache_touch", "lora_tier_cache_resident", "lora_tier_sim", "lora_pool_load_async",
           "lora_pool_unload_async", "lora_pool_prefetch", "lora_quantize_e4m3",
           "lora_layer_forward_fp8_workspace_size", "lora_layer_forward_fp8", "lora_w4_matvec", "lora_kv_append",
           "lora_tree_attention_workspace_size", "lora_tree_attention", "lora_kv_append_axes",
           "lora_tree_attention_weights_workspace_size", "lora_tree_attention_weights", "lora_kv_evict"]

if not os.path.exists(_build.LIB):
    raise ImportError(f"CUDA library {_build.LIB} is not built: run segmented_gathered_rank_gb300.build.build()")

LIB_PATH = _build.LIB
_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("lora_pool_create", _I, ctypes.POINTER(_P), _I, _I, _I, _I, _I, _I)
_sig("lora_pool_destroy", _I, _P)
_sig("lora_pool_load", _I, _P, _I, _I, _I, ctypes.c_float, _I, _I, _P, _P, _P)
_sig("lora_pool_unload", _I, _P, _I, _I)
_sig("lora_pool_free_pages", _I, _P)
_sig("lora_sgmv_shrink", _I, _P, _I, _P, _P, _I, _P, _P, _I, _I, _P)
_sig("lora_sgmv_expand", _I, _P, _I, _P, _I, _P, _P, _P, _I, _I, _P)
_sig("lora_bgmv", _I, _P, _I, _P, _P, _P, _I, _P)
_sig("lora_layer_forward_workspace_size", ctypes.c_size_t, _P, _I, _I, _I)
_sig("lora_layer_forward", _I, _P, _I, _P, _P, _P, _P, _P, _I, _I, _P, ctypes.c_size_t, _P)
_sig("lora_layer_forward_noalloc", _I, _P, _I, _P, _P, _P, _P, _P, _I, _I, _P)
_sig("lora_get_error", _I, _P, ctypes.POINTER(_I))
_sig("lora_strerror", ctypes.c_char_p, _I)
_sig("lora_launch_count", ctypes.c_ulonglong)


class AdapterSrc(ctypes.Structure):
    """``lora_adapter_src``: one entry of a prefetch list."""
    _fields_ = [("adapter", _I), ("matrix", _I), ("rank", _I), ("scale", ctypes.c_float), ("h_in", _I),
                ("h_out", _I), ("A_T", _P), ("B", _P)]


_sig("lora_pool_load_async", _I, _P, _I, _I, _I, ctypes.c_float, _I, _I, _P, _P, _P)
_sig("lora_pool_unload_async", _I, _P, _I, _I, _P)
_sig("lora_pool_prefetch", _I, _P, ctypes.POINTER(AdapterSrc), _I, _P)
_sig("lora_quantize_e4m3", _I, _P, _I, _I, _P, _P, _P)
_sig("lora_layer_forward_fp8_workspace_size", ctypes.c_size_t, _P, _I, _I, _I)
_sig("lora_layer_forward_fp8", _I, _P, _I, _P, _P, ctypes.c_float, _P, _P, _P, _I, _I, _P, ctypes.c_size_t, _P)
_sig("lora_tier_cache_create", _I, ctypes.POINTER(_P), _I, _I, _I)
_sig("lora_tier_cache_destroy", _I, _P)
_sig("lora_tier_cache_touch", _I, _P, _I, ctypes.POINTER(_I))
_sig("lora_tier_cache_resident", _I, _P, _I)
_sig("lora_tier_sim", _I, _P, ctypes.c_longlong, _I, _I, _I, ctypes.POINTER(ctypes.c_longlong))


class KvPages(ctypes.Structure):
    """``lora_kv_pages``: one layer's paged key/value cache in two CUDA tensors
    of shape [n_pages, n_kv_heads, page_size, head_dim] (kept alive by this
    object), with an optional int32 status tensor."""
    _fields_ = [("dtype", _I), ("n_pages", _I), ("page_size", _I), ("n_kv_heads", _I), ("head_dim", _I), ("k", _P),
                ("v", _P), ("status", _P)]

    def __init__(self, dtype, k_pages, v_pages, n_pages, page_size, n_kv_heads, head_dim, status=None):
        for t in (k_pages, v_pages):
            if t.numel() != n_pages * n_kv_heads * page_size * head_dim:
                raise ValueError("a cache tensor does not hold n_pages x n_kv_heads x page_size x head_dim elements")
        super().__init__(dtype, n_pages, page_size, n_kv_heads, head_dim, _dptr(k_pages), _dptr(v_pages),
                         _dptr(status))
        self.tensors = (k_pages, v_pages, status)
        self.slots = n_pages * n_kv_heads * page_size       # keys, values, weights
        self.address = ctypes.addressof(self)      # what calls pass: no reference, so no cycle, and quick


_sig("lora_w4_matvec", _I, _I, _P, _I, _I, _P, _P, _P, _I, _I, _P, _P)
_sig("lora_kv_append", _I, _P, _P, _I, _P, _I, _P, _I, _I, _I, _P, _P, _P, _I, _I, _I, _P, _P,
     ctypes.c_float, _P, _P)
# The calls of a bounded cache take a struct, packed here: their arguments one by one take ctypes longer than a launch.
_AXES = struct.Struct("@9P9if128s")             # lora_append_axes
_WEIGHTS = struct.Struct("@8PN5i2f4x")          # lora_attention_weights
_EVICTION = struct.Struct("@7P5i4x")            # lora_eviction
_sig("lora_kv_append_axes", _I, _P, ctypes.c_char_p, _P)
_sig("lora_tree_attention_weights_workspace_size", ctypes.c_size_t, _P, _I, _I, _I, _I)
_sig("lora_tree_attention_weights", _I, _P, ctypes.c_char_p, _P)
_sig("lora_kv_evict", _I, _P, ctypes.c_char_p, _P)
_sig("lora_tree_attention_workspace_size", ctypes.c_size_t, _P, _I, _I, _I)
_sig("lora_tree_attention", _I, _P, _P, _I, _P, _I, _I, _P, _P, _I, _P, _I, ctypes.c_float, _P, _P,
     ctypes.c_size_t, _P)


class LoraError(RuntimeError):
    def __init__(self, status: int, where: str, device_status: int = 0):
        self.status = status
        self.device_status = device_status
        msg = f"{where}: {lora_strerror(status)} ({status})"
        if device_status:
            msg += f", device status 0x{device_status:x}"
        super().__init__(msg)


def _check(rc: int, where: str):
    if rc != LORA_OK:
        raise LoraError(rc, where)


def _dptr(t):
    """Device pointer of a CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _ptr(t):
    """_dptr as a plain integer (cheaper to pass; decode calls are short)."""
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("expected a contiguous CUDA tensor")
    return t.data_ptr()


def _rows(t):
    """(pointer, elements between rows) of a CUDA matrix whose rows are contiguous."""
    if t is None:
        return None, 0
    if not (t.is_cuda and t.dim() == 2 and t.stride(1) == 1):
        raise ValueError("expected a CUDA matrix with contiguous rows")
    # a single row's stride means nothing, and need not be the width (a transposed column's is 1)
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld > 0x7fffffff:
        raise ValueError("rows are further apart than an int says")
    return t.data_ptr(), ld


def _address(t):
    """_ptr for a packed struct: NULL is 0."""
    if t is None:
        return 0
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("expected a contiguous CUDA tensor")
    return t.data_ptr()


def _matrix(t):
    """_rows for a packed struct, with one look at the strides."""
    if t is None:
        return 0, 0
    strides = t.stride()
    if not (t.is_cuda and len(strides) == 2 and strides[1] == 1):
        raise ValueError("expected a CUDA matrix with contiguous rows")
    rows, width = t.shape
    ld = strides[0] if rows > 1 else width      # a single row's stride means nothing
    if ld > 0x7fffffff:
        raise ValueError("rows are further apart than an int says")
    return t.data_ptr(), ld


def _hptr(a):
    """Host pointer of a numpy array or CPU tensor (kept alive by the caller)."""
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        if not a.flags.c_contiguous:
            raise ValueError("expected a C-contiguous host array")
        return ctypes.c_void_p(a.ctypes.data)
    if a.is_cuda or not a.is_contiguous():
        raise ValueError("expected a contiguous CPU tensor")
    return ctypes.c_void_p(a.data_ptr())


_raw_stream = None      # torch's current stream as an address: the Stream object around it takes longer to make than a launch


def _stream_ptr(stream):
    """Address of a stream (None: torch's current one)."""
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
            torch.cuda.current_stream()      # initialises CUDA, or says why not
            _raw_stream = ((lambda: get(device())) if get and device else
                           (lambda: torch.cuda.current_stream().cuda_stream))
        return _raw_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _stream(stream):
    return ctypes.c_void_p(_stream_ptr(stream))


def lora_strerror(status: int) -> str:
    return _lib.lora_strerror(int(status)).decode()


def lora_launch_count() -> int:
    return int(_lib.lora_launch_count())


def lora_pool_create(dtype: int, page_elems: int, n_pages: int, max_rank: int, n_matrices: int,
                     max_adapters: int) -> int:
    """Returns the pool handle (an opaque address)."""
    h = ctypes.c_void_p()
    _check(_lib.lora_pool_create(ctypes.byref(h), dtype, page_elems, n_pages, max_rank, n_matrices,
                                 max_adapters), "lora_pool_create")
    return h.value


def lora_pool_destroy(pool) -> None:
    _check(_lib.lora_pool_destroy(pool), "lora_pool_destroy")


def lora_pool_load(pool, adapter: int, matrix: int, rank: int, scale: float, h_in: int, h_out: int,
                   A_T, B, stream=None) -> None:
    _check(_lib.lora_pool_load(pool, adapter, matrix, rank, float(scale), h_in, h_out, _hptr(A_T), _hptr(B),
                               _stream(stream)), "lora_pool_load")


def lora_pool_unload(pool, adapter: int, matrix: int) -> None:
    _check(_lib.lora_pool_unload(pool, adapter, matrix), "lora_pool_unload")


def lora_pool_load_async(pool, adapter: int, matrix: int, rank: int, scale: float, h_in: int, h_out: int,
                         A_T, B, stream=None) -> None:
    """Enqueue an upload on ``stream`` and return (the host arrays are copied
    before the call returns)."""
    _check(_lib.lora_pool_load_async(pool, adapter, matrix, rank, float(scale), h_in, h_out, _hptr(A_T), _hptr(B),
                                     _stream(stream)), "lora_pool_load_async")


def lora_pool_unload_async(pool, adapter: int, matrix: int, stream=None) -> None:
    _check(_lib.lora_pool_unload_async(pool, adapter, matrix, _stream(stream)), "lora_pool_unload_async")


def lora_pool_prefetch(pool, entries, stream=None) -> int:
    """Upload every (adapter, matrix, rank, scale, h_in, h_out, A_T, B) entry not
    resident yet; returns how many uploads were enqueued."""
    entries = list(entries)
    arr = (AdapterSrc * max(1, len(entries)))()
    for i, (a, m, r, sc, hi, ho, at, b) in enumerate(entries):
        arr[i] = AdapterSrc(a, m, r, float(sc), hi, ho, _hptr(at), _hptr(b))
    rc = _lib.lora_pool_prefetch(pool, arr, len(entries), _stream(stream))
    if rc < 0:
        raise LoraError(rc, "lora_pool_prefetch")
    return int(rc)


def lora_pool_free_pages(pool) -> int:
    return int(_lib.lora_pool_free_pages(pool))


def lora_sgmv_shrink(pool, matrix, x, v, ld_v, seg_starts, seg_adapter, S, T, stream=None) -> None:
    _check(_lib.lora_sgmv_shrink(pool, matrix, _dptr(x), _dptr(v), ld_v, _dptr(seg_starts), _dptr(seg_adapter),
                                 S, T, _stream(stream)), "lora_sgmv_shrink")


def lora_sgmv_expand(pool, matrix, v, ld_v, y, seg_starts, seg_adapter, S, T, stream=None) -> None:
    _check(_lib.lora_sgmv_expand(pool, matrix, _dptr(v), ld_v, _dptr(y), _dptr(seg_starts), _dptr(seg_adapter),
                                 S, T, _stream(stream)), "lora_sgmv_expand")


def lora_bgmv(pool, matrix, x, y, token_adapter, T, stream=None) -> None:
    _check(_lib.lora_bgmv(pool, matrix, _dptr(x), _dptr(y), _dptr(token_adapter), T, _stream(stream)),
           "lora_bgmv")


def lora_layer_forward_workspace_size(pool, matrix, S, T) -> int:
    return int(_lib.lora_layer_forward_workspace_size(pool, matrix, S, T))


def lora_layer_forward(pool, matrix, x, W, y, seg_starts, seg_adapter, S, T, workspace, ws_bytes=None,
                       stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib.lora_layer_forward(pool, matrix, _dptr(x), _dptr(W), _dptr(y), _dptr(seg_starts),
                                   _dptr(seg_adapter), S, T, _dptr(workspace), ws_bytes, _stream(stream)),
           "lora_layer_forward")


def lora_layer_forward_noalloc(pool, matrix, x, W, y, seg_starts, seg_adapter, S, T, stream=None) -> None:
    """lora_layer_forward with the library's fixed scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    _check(_lib.lora_layer_forward_noalloc(pool, matrix, _dptr(x), _dptr(W), _dptr(y), _dptr(seg_starts),
                                           _dptr(seg_adapter), S, T, _stream(stream)),
           "lora_layer_forward_noalloc")


def lora_get_error(pool) -> tuple[int, int]:
    """(status, device status word); the word is cleared."""
    word = ctypes.c_int(0)
    rc = _lib.lora_get_error(pool, ctypes.byref(word))
    return int(rc), int(word.value)


def lora_tier_cache_create(n_keys: int, gpu_slots: int, host_slots: int) -> int:
    """Two-tier LRU residency cache (host only); returns its handle."""
    h = ctypes.c_void_p()
    _check(_lib.lora_tier_cache_create(ctypes.byref(h), n_keys, gpu_slots, host_slots), "lora_tier_cache_create")
    return h.value


def lora_tier_cache_destroy(cache) -> None:
    _check(_lib.lora_tier_cache_destroy(cache), "lora_tier_cache_destroy")


def lora_tier_cache_touch(cache, adapter: int) -> tuple[int, int]:
    """(tier that served the request, adapter the GPU tier evicted or -1)."""
    ev = ctypes.c_int(-1)
    rc = _lib.lora_tier_cache_touch(cache, adapter, ctypes.byref(ev))
    if rc < 0:
        raise LoraError(rc, "lora_tier_cache_touch")
    return int(rc), int(ev.value)


def lora_tier_cache_resident(cache, adapter: int) -> int:
    rc = _lib.lora_tier_cache_resident(cache, adapter)
    if rc < 0:
        raise LoraError(rc, "lora_tier_cache_resident")
    return int(rc)


def lora_tier_sim(trace, n_keys: int, gpu_slots: int, host_slots: int) -> tuple[int, int, int]:
    """(GPU hits, host hits, disk loads) of a request trace (int32 host array)."""
    tr = np.ascontiguousarray(trace, np.int32)
    counts = (ctypes.c_longlong * 3)()
    _check(_lib.lora_tier_sim(ctypes.c_void_p(tr.ctypes.data), len(tr), n_keys, gpu_slots, host_slots, counts),
           "lora_tier_sim")
    return int(counts[0]), int(counts[1]), int(counts[2])


def lora_quantize_e4m3(x, T, h, q, sx, stream=None) -> None:
    """Per-row e4m3 codes (uint8 tensor) and fp32 scales of a bf16 tensor."""
    _check(_lib.lora_quantize_e4m3(_dptr(x), T, h, _dptr(q), _dptr(sx), _stream(stream)), "lora_quantize_e4m3")


def lora_layer_forward_fp8_workspace_size(pool, matrix, S, T) -> int:
    return int(_lib.lora_layer_forward_fp8_workspace_size(pool, matrix, S, T))


def lora_layer_forward_fp8(pool, matrix, x, W8, w_scale, y, seg_starts, seg_adapter, S, T, workspace, ws_bytes=None,
                           stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib.lora_layer_forward_fp8(pool, matrix, _dptr(x), _dptr(W8), float(w_scale), _dptr(y),
                                       _dptr(seg_starts), _dptr(seg_adapter), S, T, _dptr(workspace), ws_bytes,
                                       _stream(stream)), "lora_layer_forward_fp8")


def lora_w4_matvec(dtype, x, T, h_in, codes, scales, zeros, group, h_out, y, stream=None) -> None:
    """Products with 4-bit weights (uint8 codes, bf16 scales, uint8 zeros or None); y is overwritten."""
    rc = _lib.lora_w4_matvec(dtype, _ptr(x), T, h_in, _ptr(codes), _ptr(scales), _ptr(zeros), group, h_out, _ptr(y),
                             _stream_ptr(stream))
    if rc:
        _check(rc, "lora_w4_matvec")


def lora_kv_append(kv, q, k, v, T, n_q_heads, positions, slots, cos_sin, n_pos, rot_dim, interleaved, q_out,
                   q_norm=None, k_norm=None, eps=1e-6, stream=None) -> None:
    """Norm, rotation and append of T tokens; q, k and v are matrices of T rows (any row stride), slots int64."""
    (pq, ld_q), (pk, ld_k), (pv, ld_v) = _rows(q), _rows(k), _rows(v)
    rc = _lib.lora_kv_append(kv.address, pq, ld_q, pk, ld_k, pv, ld_v, T, n_q_heads, _ptr(positions), _ptr(slots),
                             _ptr(cos_sin), n_pos, rot_dim, 1 if interleaved else 0, _ptr(q_norm), _ptr(k_norm), eps,
                             _ptr(q_out), _stream_ptr(stream))
    if rc:
        _check(rc, "lora_kv_append")


def lora_kv_append_axes(kv, q, k, v, T, n_q_heads, positions, n_axes, pair_axis, slots, cos_sin, n_pos, rot_dim, interleaved,
                        q_out, q_norm=None, k_norm=None, eps=1e-6, stream=None) -> None:
    """lora_kv_append with n_axes positions a token (int32 [T, n_axes]); pair_axis: the axis of each rotated pair, as
    bytes (quickest) or a sequence of whole numbers."""
    (pq, ld_q), (pk, ld_k), (pv, ld_v) = _matrix(q), _matrix(k), _matrix(v)
    if type(pair_axis) is not bytes:
        pair_axis = bytes(list(pair_axis))
    if len(pair_axis) < rot_dim // 2:
        raise ValueError("pair_axis names fewer pairs than rot_dim has")
    args = _AXES.pack(pq, pk, pv, _address(q_out), _address(positions), _address(slots), _address(cos_sin), _address(q_norm),
                      _address(k_norm), ld_q, ld_k, ld_v, T, n_q_heads, n_axes, n_pos, rot_dim, 1 if interleaved else 0, eps, pair_axis)
    rc = _lib.lora_kv_append_axes(kv.address, args, _stream_ptr(stream))
    if rc:
        _check(rc, "lora_kv_append_axes")


def lora_tree_attention_workspace_size(kv, n_q_heads, S, T) -> int:
    return int(_lib.lora_tree_attention_workspace_size(kv.address, n_q_heads, S, T))


def lora_tree_attention(kv, q, n_q_heads, seg_starts, S, T, kv_lens, page_table, max_pages, tree_mask, mask_words, scale,
                        out, workspace, ws_bytes=None, stream=None) -> None:
    """Attention of drafted tokens over the cache; tree_mask is int64 [T, mask_words], or None for causal chains."""
    if ws_bytes is None:
        ws_bytes = workspace.nbytes
    rc = _lib.lora_tree_attention(kv.address, _ptr(q), n_q_heads, _ptr(seg_starts), S, T, _ptr(kv_lens), _ptr(page_table),
                                  max_pages, _ptr(tree_mask), mask_words, scale, _ptr(out), _ptr(workspace), ws_bytes,
                                  _stream_ptr(stream))
    if rc:
        _check(rc, "lora_tree_attention")


def _plane(kv, t):
    """Pointer of one fp32 number a slot and kv head of the cache."""
    if t is not None and t.numel() < kv.slots:
        raise ValueError("expected n_pages x n_kv_heads x page_size numbers")
    return _address(t)


def lora_tree_attention_weights_workspace_size(kv, n_q_heads, S, T, max_pages) -> int:
    return int(_lib.lora_tree_attention_weights_workspace_size(kv.address, n_q_heads, S, T, max_pages))


def lora_tree_attention_weights(kv, weights, decay, q, n_q_heads, seg_starts, S, T, kv_lens, page_table, max_pages, tree_mask,
                                mask_words, scale, out, workspace, ws_bytes=None, stream=None) -> None:
    """lora_tree_attention that adds the weight of each cached token, times decay what it had, to weights (float
    [n_pages, n_kv_heads, page_size]).  A workspace below its size, down to that for max_pages 0, takes longer."""
    if ws_bytes is None:
        ws_bytes = workspace.nbytes
    args = _WEIGHTS.pack(_plane(kv, weights), _address(q), _address(seg_starts), _address(kv_lens), _address(page_table), _address(tree_mask),
                         _address(out), _address(workspace), ws_bytes, n_q_heads, S, T, max_pages, mask_words, scale, decay)
    rc = _lib.lora_tree_attention_weights(kv.address, args, _stream_ptr(stream))
    if rc:
        _check(rc, "lora_tree_attention_weights")


def lora_kv_evict(kv, scores, weights, S, kv_lens, page_table, max_pages, keep, first, recent, kept, ld_kept, new_lens,
                  stream=None) -> None:
    """Every kv head keeps its keep[s] tokens of the greatest scores (float [n_pages, n_kv_heads, page_size]), in order;
    weights (None, scores itself or another such tensor) move along; kept gets the indices, new_lens the lengths."""
    if kept is not None and kept.numel() < S * kv.n_kv_heads * ld_kept:
        raise ValueError("kept does not hold S x n_kv_heads x ld_kept indices")
    args = _EVICTION.pack(_plane(kv, scores), _plane(kv, weights), _address(kv_lens), _address(page_table), _address(keep), _address(kept),
                          _address(new_lens), S, max_pages, first, recent, ld_kept)
    rc = _lib.lora_kv_evict(kv.address, args, _stream_ptr(stream))
    if rc:
        _check(rc, "lora_kv_evict")
