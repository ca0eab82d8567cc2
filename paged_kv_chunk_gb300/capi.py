"""Python binding of the C ABI in ``include/oasr_attn.h`` (``liboasr_attn.so``).

Argument marshalling only: each function checks that the torch tensors it is given
live on the current CUDA device with the layout the C ABI documents, derives the
sizes from their shapes and passes raw device pointers plus the current CUDA stream.
Every step of the computation runs in the library's CUDA kernels; there is no other
path, and a missing library raises instead of falling back.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liboasr_attn.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "oasr_attn.h")

OASR_OK, OASR_ERR_INVALID_ARG, OASR_ERR_UNSUPPORTED, OASR_ERR_CUDA = 0, 1, 2, 3
OASR_ERR_BOUNDS, OASR_ERR_TIMEOUT = 4, 5
OASR_F32, OASR_BF16 = 0, 1
STATUS_BOUNDS_BIT, STATUS_TIMEOUT_BIT = 1, 2

_lock = threading.Lock()
_lib = None


class OasrError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load liboasr_attn.so (built by ``paged_kv_chunk_gb300.build``); raise if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m paged_kv_chunk_gb300.build`"
                               " (or __graft_entry__.build()) first")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
        L.oasr_paged_append.argtypes = [P, P, P, P, I, I, P, I, P, I, I, I, I, I, S]
        L.oasr_chunk_relattn_paged.argtypes = [P, P, P, I, I, P, I, P, P, P, P, I, P, I, I, I, I,
                                               F, I, S]
        L.oasr_chunk_step_paged.argtypes = [P, P, P, P, P, I, I, P, I, P, P, P, P, I, P, I, I, I,
                                            I, F, I, S]
        L.oasr_packed_relattn_varlen.argtypes = [P, P, P, P, I, I, I, P, P, P, I, P, I, I, F, I, S]
        L.oasr_packed_relattn_chunked.argtypes = [P, P, P, P, I, I, I, P, P, P, I, P, I, I, F, I, I,
                                                  I, S]
        L.oasr_window_commit.argtypes = [P, P, I, I, I, I, I, S]
        L.oasr_project_qkv_pos.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, S]
        L.oasr_paged_append_e4m3.argtypes = [P, P, P, P, P, I, I, P, I, P, I, I, I, I, I, S]
        L.oasr_paged_read_e4m3.argtypes = [P, P, P, I, I, P, I, P, P, P, P, I, I, I, I, I, S]
        L.oasr_chunk_relattn_paged_e4m3.argtypes = [P, P, P, P, I, I, P, I, P, P, P, P, I, P, I, I,
                                                    I, I, F, I, S]
        L.oasr_chunk_step_paged_e4m3.argtypes = [P, P, P, P, P, P, I, I, P, I, P, P, P, P, I, P, I,
                                                 I, I, I, F, I, S]
        L.oasr_quantize_rows.argtypes = [P, P, P, I, I, I, S]
        L.oasr_linear_w8a8.argtypes = [P, P, P, P, P, P, I, I, I, I, S]
        L.oasr_project_qkv_pos_w8a8.argtypes = [P] * 13 + [I, I, I, I, I, S]
        Q = ctypes.c_int64
        L.oasr_block_table_update.argtypes = [P, P, P, I, I, I, P, I, P, P, I, P, S]
        L.oasr_paged_append_slots.argtypes = [P, P, Q, Q, P, P, I, I, P, I, I, I, I, S]
        L.oasr_cross_attn_packed.argtypes = [P, Q, P, Q, P, Q, P, P, I, I, I, I, I, P, I, I, I, F, I, S]
        L.oasr_cross_attn_paged.argtypes = [P, Q, P, P, I, I, P, I, P, P, I, I, I, I, P, I, I, I, F, I, S]
        L.oasr_quantize_blocks.argtypes = [P, P, P, I, I, I, S]
        L.oasr_linear_e4m3.argtypes = [P, P, P, P, P, P, I, I, I, I, S]
        for fn in ("oasr_block_table_update", "oasr_paged_append_slots", "oasr_cross_attn_packed",
                   "oasr_cross_attn_paged", "oasr_quantize_blocks", "oasr_linear_e4m3",
                   "oasr_quantize_rows", "oasr_linear_w8a8", "oasr_project_qkv_pos_w8a8",
                   "oasr_paged_append_e4m3", "oasr_paged_read_e4m3",
                   "oasr_chunk_relattn_paged_e4m3", "oasr_chunk_step_paged_e4m3",
                   "oasr_paged_append", "oasr_chunk_relattn_paged", "oasr_chunk_step_paged",
                   "oasr_packed_relattn_varlen", "oasr_packed_relattn_chunked",
                   "oasr_window_commit", "oasr_project_qkv_pos"):
            getattr(L, fn).restype = I
        L.oasr_status_string.argtypes = [I]
        L.oasr_status_string.restype = ctypes.c_char_p
        L.oasr_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), I]
        L.oasr_device_status.restype = I
        L.oasr_version.argtypes = []
        L.oasr_version.restype = I
        L.oasr_selftest_wait.argtypes = [ctypes.c_uint, S]
        L.oasr_selftest_wait.restype = I
        _lib = L
        return L


def header_symbols() -> list[str]:
    """Names of the functions ``include/oasr_attn.h`` declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(oasr_[a-z0-9_]+)\s*\(", text)))


# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _check(fn: str, status: int):
    if status != OASR_OK:
        msg = load().oasr_status_string(status).decode()
        raise OasrError(fn, status, msg)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return OASR_BF16
    if t.dtype == torch.float32:
        return OASR_F32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or float32")


def _dev(t: torch.Tensor, name: str, dtype=None, ndim=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        # the kernels run on the current device: another device's pointer would be a fault
        raise ValueError(f"{name} is on {t.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def oasr_paged_append(k_new, v_new, k_pool, v_pool, block_table, cache_seqlens, stream=None):
    """Write the chunk (k_new, v_new [B,T,H,D]) into the pools [nb,bs,H,D] in place."""
    L = load()
    dt = _dtype_code(k_new)
    B, T, H, D = k_new.shape
    nb, bs = k_pool.shape[:2]
    if tuple(v_new.shape) != (B, T, H, D) or tuple(k_pool.shape[2:]) != (H, D) \
            or v_pool.shape != k_pool.shape:
        raise ValueError("shape mismatch between chunk and pools")
    if tuple(block_table.shape[:1]) != (B,) or tuple(cache_seqlens.shape) != (B,):
        raise ValueError("block_table must be [B, mbps] and cache_seqlens [B]")
    _check("oasr_paged_append", L.oasr_paged_append(
        _dev(k_new, "k_new", k_new.dtype, 4), _dev(v_new, "v_new", k_new.dtype, 4),
        _dev(k_pool, "k_pool", k_new.dtype, 4), _dev(v_pool, "v_pool", k_new.dtype, 4), nb, bs,
        _dev(block_table, "block_table", torch.int32, 2), block_table.shape[1],
        _dev(cache_seqlens, "cache_seqlens", torch.int32, 1), B, T, H, D, dt, _stream(stream)))


def _chunk_common(q, k_pool, v_pool, block_table, cache_seqlens, pos_bias_u, pos_bias_v, rel,
                  out):
    B, T, H, D = q.shape
    if k_pool.dim() != 4 or tuple(k_pool.shape[2:]) != (H, D):
        raise ValueError("k_pool must be [num_blocks, block_size, H, D]")
    if v_pool.shape != k_pool.shape:
        raise ValueError("v_pool must have k_pool's shape")
    if tuple(pos_bias_u.shape) != (H, D) or tuple(pos_bias_v.shape) != (H, D):
        raise ValueError("pos biases must be [H, D]")
    if rel.dim() != 3 or tuple(rel.shape[1:]) != (H, D):
        raise ValueError("rel must be [R, H, D]")
    if tuple(out.shape) != (B, T, H, D) or out.dtype != q.dtype:
        raise ValueError("out must be [B, T, H, D] of q's dtype")
    if block_table.dim() != 2 or block_table.shape[0] != B or tuple(cache_seqlens.shape) != (B,):
        raise ValueError("block_table must be [B, mbps] and cache_seqlens [B]")
    return B, T, H, D


def oasr_chunk_relattn_paged(q, k_pool, v_pool, block_table, cache_seqlens, pos_bias_u,
                             pos_bias_v, rel, out=None, scale=None, stream=None):
    """Streaming chunk attention over the paged pool; returns out [B,T,H,D]."""
    L = load()
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    B, T, H, D = _chunk_common(q, k_pool, v_pool, block_table, cache_seqlens, pos_bias_u,
                               pos_bias_v, rel, out)
    scale = D ** -0.5 if scale is None else float(scale)
    _check("oasr_chunk_relattn_paged", L.oasr_chunk_relattn_paged(
        _dev(q, "q", q.dtype), _dev(k_pool, "k_pool", q.dtype), _dev(v_pool, "v_pool", q.dtype),
        k_pool.shape[0], k_pool.shape[1], _dev(block_table, "block_table", torch.int32),
        block_table.shape[1], _dev(cache_seqlens, "cache_seqlens", torch.int32),
        _dev(pos_bias_u, "pos_bias_u", q.dtype), _dev(pos_bias_v, "pos_bias_v", q.dtype),
        _dev(rel, "rel", q.dtype), rel.shape[0], _dev(out, "out", q.dtype), B, T, H, D, scale, dt,
        _stream(stream)))
    return out


def oasr_chunk_step_paged(q, k_new, v_new, k_pool, v_pool, block_table, cache_seqlens,
                          pos_bias_u, pos_bias_v, rel, out=None, scale=None, stream=None):
    """Fused append + streaming chunk attention; returns out [B,T,H,D]."""
    L = load()
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    B, T, H, D = _chunk_common(q, k_pool, v_pool, block_table, cache_seqlens, pos_bias_u,
                               pos_bias_v, rel, out)
    if tuple(k_new.shape) != (B, T, H, D) or tuple(v_new.shape) != (B, T, H, D):
        raise ValueError("k_new, v_new must be [B, T, H, D]")
    scale = D ** -0.5 if scale is None else float(scale)
    _check("oasr_chunk_step_paged", L.oasr_chunk_step_paged(
        _dev(q, "q", q.dtype), _dev(k_new, "k_new", q.dtype), _dev(v_new, "v_new", q.dtype),
        _dev(k_pool, "k_pool", q.dtype), _dev(v_pool, "v_pool", q.dtype), k_pool.shape[0],
        k_pool.shape[1], _dev(block_table, "block_table", torch.int32), block_table.shape[1],
        _dev(cache_seqlens, "cache_seqlens", torch.int32), _dev(pos_bias_u, "pos_bias_u", q.dtype),
        _dev(pos_bias_v, "pos_bias_v", q.dtype), _dev(rel, "rel", q.dtype), rel.shape[0],
        _dev(out, "out", q.dtype), B, T, H, D, scale, dt, _stream(stream)))
    return out


def oasr_packed_relattn_varlen(q, k, v, cu_seqlens, max_seqlen, pos_bias_u, pos_bias_v, rel,
                               out=None, scale=None, stream=None):
    """Packed varlen bidirectional rel-pos attention; returns out [total,H,D]."""
    L = load()
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    total, H, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or out.shape != q.shape:
        raise ValueError("q, k, v, out must share their shape [total, H, D]")
    if tuple(pos_bias_u.shape) != (H, D) or tuple(pos_bias_v.shape) != (H, D):
        raise ValueError("pos biases must be [H, D]")
    if rel.dim() != 3 or tuple(rel.shape[1:]) != (H, D):
        raise ValueError("rel must be [R, H, D]")
    scale = D ** -0.5 if scale is None else float(scale)
    _check("oasr_packed_relattn_varlen", L.oasr_packed_relattn_varlen(
        _dev(q, "q", q.dtype), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype),
        _dev(cu_seqlens, "cu_seqlens", torch.int32, 1), cu_seqlens.shape[0] - 1, int(max_seqlen),
        total, _dev(pos_bias_u, "pos_bias_u", q.dtype), _dev(pos_bias_v, "pos_bias_v", q.dtype),
        _dev(rel, "rel", q.dtype), rel.shape[0], _dev(out, "out", q.dtype), H, D, scale, dt,
        _stream(stream)))
    return out


def oasr_packed_relattn_chunked(q, k, v, cu_seqlens, max_seqlen, pos_bias_u, pos_bias_v, rel,
                                chunk_size, left_chunks, out=None, scale=None, stream=None):
    """Chunked-limited packed attention (own chunk + left_chunks earlier chunks per query);
    returns out [total,H,D]."""
    L = load()
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    total, H, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or out.shape != q.shape:
        raise ValueError("q, k, v, out must share their shape [total, H, D]")
    if tuple(pos_bias_u.shape) != (H, D) or tuple(pos_bias_v.shape) != (H, D):
        raise ValueError("pos biases must be [H, D]")
    if rel.dim() != 3 or tuple(rel.shape[1:]) != (H, D):
        raise ValueError("rel must be [R, H, D]")
    scale = D ** -0.5 if scale is None else float(scale)
    _check("oasr_packed_relattn_chunked", L.oasr_packed_relattn_chunked(
        _dev(q, "q", q.dtype), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype),
        _dev(cu_seqlens, "cu_seqlens", torch.int32, 1), cu_seqlens.shape[0] - 1, int(max_seqlen),
        total, _dev(pos_bias_u, "pos_bias_u", q.dtype), _dev(pos_bias_v, "pos_bias_v", q.dtype),
        _dev(rel, "rel", q.dtype), rel.shape[0], _dev(out, "out", q.dtype), H, D, scale,
        int(chunk_size), int(left_chunks), dt, _stream(stream)))
    return out


def oasr_window_commit(block_table, cache_seqlens, T, block_size, window_frames, stream=None):
    """Commit a step's chunk with fixed-window history eviction, in place on the device:
    rotates each full stream's block-table row and advances cache_seqlens."""
    L = load()
    if block_table.dim() != 2 or cache_seqlens.dim() != 1 or cache_seqlens.shape[0] != block_table.shape[0]:
        raise ValueError("block_table must be [B, max_blocks_per_seq] and cache_seqlens [B]")
    B, mbps = block_table.shape
    _check("oasr_window_commit", L.oasr_window_commit(
        _dev(block_table, "block_table", torch.int32, 2), _dev(cache_seqlens, "cache_seqlens", torch.int32, 1),
        B, mbps, int(block_size), int(T), int(window_frames), _stream(stream)))


def oasr_project_qkv_pos(x, w_qkv, b_qkv, pos_emb, w_pos, H, q=None, k=None, v=None, rel=None,
                         stream=None):
    """q, k, v = x . w_qkv^T + b_qkv (split in three, [M, H, 64] each) and
    rel = pos_emb . w_pos^T ([R, H, 64]), bf16, one launch; returns (q, k, v, rel)."""
    L = load()
    M, d = x.shape
    R = pos_emb.shape[0]
    if tuple(w_qkv.shape) != (3 * d, d) or tuple(b_qkv.shape) != (3 * d,) or \
            tuple(w_pos.shape) != (d, d) or pos_emb.dim() != 2 or pos_emb.shape[1] != d or d % H:
        raise ValueError("shapes: x [M,d], w_qkv [3d,d], b_qkv [3d], pos_emb [R,d], w_pos [d,d]")
    D = d // H
    q = torch.empty((M, H, D), dtype=x.dtype, device=x.device) if q is None else q
    k = torch.empty((M, H, D), dtype=x.dtype, device=x.device) if k is None else k
    v = torch.empty((M, H, D), dtype=x.dtype, device=x.device) if v is None else v
    rel = torch.empty((R, H, D), dtype=x.dtype, device=x.device) if rel is None else rel
    if any(tuple(t.shape) != (M, H, D) for t in (q, k, v)) or tuple(rel.shape) != (R, H, D):
        raise ValueError("q, k, v must be [M, H, d/H] and rel [R, H, d/H]")
    _check("oasr_project_qkv_pos", L.oasr_project_qkv_pos(
        _dev(x, "x", x.dtype, 2), _dev(w_qkv, "w_qkv", x.dtype, 2), _dev(b_qkv, "b_qkv", x.dtype, 1),
        _dev(pos_emb, "pos_emb", x.dtype, 2), _dev(w_pos, "w_pos", x.dtype, 2),
        _dev(q, "q", x.dtype), _dev(k, "k", x.dtype), _dev(v, "v", x.dtype), _dev(rel, "rel", x.dtype),
        M, R, d, H, _dtype_code(x), _stream(stream)))
    return q, k, v, rel


def _good(device, dtype, *tensors) -> bool:
    """Whether the tensors are what `_dev` asks for: contiguous, of the dtype, on the device.  It runs
    on every call, so it makes do with the attribute reads that tell."""
    try:
        for t in tensors:
            if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
                return False
    except AttributeError:
        return False
    return True


def _refuse(**named):
    """Raise what `_dev` finds wrong with the first bad (tensor, dtype)."""
    for name, (t, dtype) in named.items():
        _dev(t, name, dtype)
    raise ValueError("tensors on another device than the current one")


_DTYPES = {torch.float32: OASR_F32, torch.bfloat16: OASR_BF16}


def _code(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: bf16 or float32")
    return code


def _fits(*sizes):
    """Sizes reach the library as C ints, which ctypes would cut off without a word."""
    if max(sizes) > 0x7fffffff:
        raise ValueError("sizes must be below 2^31")


def _lib_device():
    """The library and the current device (-2 without one: no tensor is on it)."""
    try:
        return _lib or load(), torch._C._cuda_getDevice()
    except RuntimeError:
        if _lib is None:
            raise
        return _lib, -2


def _cache_e4m3(dev, k_pool, v_pool, kv_scale, block_table, cache_seqlens, B, H, D):
    """Checks an 8-bit cache (pools [nb,H,bs,D], scales [nb,H,2,bs]) and its table; returns
    num_blocks, block_size and max_blocks_per_seq."""
    shape = k_pool.shape
    if len(shape) != 4 or shape[1] != H or shape[3] != D:
        raise ValueError("k_pool must be [num_blocks, H, block_size, D]")
    if v_pool.shape != shape:
        raise ValueError("v_pool must have k_pool's shape")
    nb, bs = shape[0], shape[2]
    if kv_scale.shape != (nb, H, 2, bs):
        raise ValueError("kv_scale must be [num_blocks, H, 2, block_size]")
    table = block_table.shape
    if len(table) != 2 or table[0] != B or cache_seqlens.shape != (B,):
        raise ValueError("block_table must be [B, mbps] and cache_seqlens [B]")
    _fits(nb, bs, table[1])
    if not (_good(dev, torch.float8_e4m3fn, k_pool, v_pool) and _good(dev, torch.uint8, kv_scale)
            and _good(dev, torch.int32, block_table, cache_seqlens)):
        _refuse(k_pool=(k_pool, torch.float8_e4m3fn), v_pool=(v_pool, torch.float8_e4m3fn),
                kv_scale=(kv_scale, torch.uint8), block_table=(block_table, torch.int32),
                cache_seqlens=(cache_seqlens, torch.int32))
    return nb, bs, table[1]


def oasr_paged_append_e4m3(k_new, v_new, k_pool, v_pool, kv_scale, block_table, cache_seqlens,
                           stream=None):
    """Quantise the chunk (k_new, v_new [B,T,H,64]) into the 8-bit pools (float8_e4m3fn
    [nb,H,bs,64]) and their scales (uint8 [nb,H,2,bs]), in place."""
    L, dev = _lib_device()
    dt = k_new.dtype
    code = _code(dt)
    B, T, H, D = k_new.shape
    if v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must share their shape [B, T, H, D]")
    nb, bs, mbps = _cache_e4m3(dev, k_pool, v_pool, kv_scale, block_table, cache_seqlens, B, H, D)
    if not _good(dev, dt, k_new, v_new):
        _refuse(k_new=(k_new, dt), v_new=(v_new, dt))
    _check("oasr_paged_append_e4m3", L.oasr_paged_append_e4m3(
        k_new.data_ptr(), v_new.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), kv_scale.data_ptr(), nb, bs,
        block_table.data_ptr(), mbps, cache_seqlens.data_ptr(), B, T, H, D, code, _stream(stream)))


def oasr_paged_read_e4m3(k_pool, v_pool, kv_scale, block_table, cache_seqlens, length, start=None,
                         k=None, v=None, dtype=torch.bfloat16, stream=None):
    """Values of each stream's positions start[b] .. start[b] + length - 1 (start None: from 0) as
    dense [B,length,H,64] tensors (k, v) of ``dtype`` (or of the k and v given); zeros past the
    cached length."""
    L, dev = _lib_device()
    B, n = block_table.shape[0], int(length)
    _, H, _, D = k_pool.shape
    if n < 1:
        raise ValueError("length must be at least 1")
    _fits(n)
    if start is not None and start.shape != (B,):
        raise ValueError("start must be [B]")
    nb, bs, mbps = _cache_e4m3(dev, k_pool, v_pool, kv_scale, block_table, cache_seqlens, B, H, D)
    shape = (B, n, H, D)
    if k is None:
        k = torch.empty(shape, dtype=dtype if v is None else v.dtype, device=k_pool.device)
    if v is None:
        v = torch.empty_like(k)
    if k.shape != shape or v.shape != shape:
        raise ValueError("k and v must be [B, length, H, D]")
    dt = k.dtype
    code = _code(dt)
    if not _good(dev, dt, k, v) or (start is not None and not _good(dev, torch.int32, start)):
        _refuse(k=(k, dt), v=(v, dt), **({} if start is None else {"start": (start, torch.int32)}))
    _check("oasr_paged_read_e4m3", L.oasr_paged_read_e4m3(
        k_pool.data_ptr(), v_pool.data_ptr(), kv_scale.data_ptr(), nb, bs, block_table.data_ptr(), mbps,
        cache_seqlens.data_ptr(), None if start is None else start.data_ptr(), k.data_ptr(), v.data_ptr(), B, n,
        H, D, code, _stream(stream)))
    return k, v


def _attention_e4m3(dev, q, pos_bias_u, pos_bias_v, rel, out, k_new=None, v_new=None):
    """Checks the attention's own tensors; returns the output, the sizes and the dtype's code."""
    shape = q.shape
    B, T, H, D = shape
    dt = q.dtype
    code = _code(dt)
    if pos_bias_u.shape != (H, D) or pos_bias_v.shape != (H, D):
        raise ValueError("pos biases must be [H, D]")
    r = rel.shape
    if len(r) != 3 or r[1] != H or r[2] != D:
        raise ValueError("rel must be [R, H, D]")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != shape or out.dtype != dt:
        raise ValueError("out must be [B, T, H, D] of q's dtype")
    if k_new is not None and (k_new.shape != shape or v_new.shape != shape):
        raise ValueError("k_new, v_new must be [B, T, H, D]")
    if not _good(dev, dt, q, pos_bias_u, pos_bias_v, rel, out, *(() if k_new is None else (k_new, v_new))):
        _refuse(q=(q, dt), pos_bias_u=(pos_bias_u, dt), pos_bias_v=(pos_bias_v, dt), rel=(rel, dt), out=(out, dt),
                **({} if k_new is None else {"k_new": (k_new, dt), "v_new": (v_new, dt)}))
    return out, B, T, H, D, r[0], code


def oasr_chunk_relattn_paged_e4m3(q, k_pool, v_pool, kv_scale, block_table, cache_seqlens,
                                  pos_bias_u, pos_bias_v, rel, out=None, scale=None, stream=None):
    """Streaming chunk attention over the 8-bit paged cache; returns out [B,T,H,64]."""
    L, dev = _lib_device()
    out, B, T, H, D, R, code = _attention_e4m3(dev, q, pos_bias_u, pos_bias_v, rel, out)
    nb, bs, mbps = _cache_e4m3(dev, k_pool, v_pool, kv_scale, block_table, cache_seqlens, B, H, D)
    _check("oasr_chunk_relattn_paged_e4m3", L.oasr_chunk_relattn_paged_e4m3(
        q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), kv_scale.data_ptr(), nb, bs, block_table.data_ptr(),
        mbps, cache_seqlens.data_ptr(), pos_bias_u.data_ptr(), pos_bias_v.data_ptr(), rel.data_ptr(), R,
        out.data_ptr(), B, T, H, D, D ** -0.5 if scale is None else scale, code, _stream(stream)))
    return out


def oasr_chunk_step_paged_e4m3(q, k_new, v_new, k_pool, v_pool, kv_scale, block_table,
                               cache_seqlens, pos_bias_u, pos_bias_v, rel, out=None, scale=None,
                               stream=None):
    """Fused append + streaming chunk attention over the 8-bit paged cache; returns out
    [B,T,H,64]."""
    L, dev = _lib_device()
    out, B, T, H, D, R, code = _attention_e4m3(dev, q, pos_bias_u, pos_bias_v, rel, out, k_new, v_new)
    nb, bs, mbps = _cache_e4m3(dev, k_pool, v_pool, kv_scale, block_table, cache_seqlens, B, H, D)
    _check("oasr_chunk_step_paged_e4m3", L.oasr_chunk_step_paged_e4m3(
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), kv_scale.data_ptr(),
        nb, bs, block_table.data_ptr(), mbps, cache_seqlens.data_ptr(), pos_bias_u.data_ptr(),
        pos_bias_v.data_ptr(), rel.data_ptr(), R, out.data_ptr(), B, T, H, D,
        D ** -0.5 if scale is None else scale, code, _stream(stream)))
    return out


def oasr_quantize_rows(x, x8=None, scale=None, stream=None):
    """Rows of x [M,K] as 8-bit integers with a scale each; returns (x8 int8 [M,K], scale
    float32 [M])."""
    L, dev = _lib_device()
    dt = x.dtype
    code = _code(dt)
    M, K = x.shape
    _fits(M, K)
    if x8 is None:
        x8 = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    if x8.shape != (M, K) or scale.shape != (M,):
        raise ValueError("x8 must be [M, K] and scale [M]")
    if not (_good(dev, dt, x) and _good(dev, torch.int8, x8) and _good(dev, torch.float32, scale)):
        _refuse(x=(x, dt), x8=(x8, torch.int8), scale=(scale, torch.float32))
    _check("oasr_quantize_rows", L.oasr_quantize_rows(
        x.data_ptr(), x8.data_ptr(), scale.data_ptr(), M, K, code, _stream(stream)))
    return x8, scale


def oasr_linear_w8a8(x8, x_scale, w8, w_scale, bias=None, out=None, out_dtype=torch.bfloat16,
                     stream=None):
    """(x8 . w8^T) * x_scale[:, None] * w_scale + bias from int8 x8 [M,K], w8 [N,K]; returns out
    [M,N] of ``out_dtype`` (or of the out given)."""
    L, dev = _lib_device()
    M, K = x8.shape
    N, Kw = w8.shape
    _fits(M, N, K)
    if Kw != K or x_scale.shape != (M,) or w_scale.shape != (N,):
        raise ValueError("shapes: x8 [M,K], x_scale [M], w8 [N,K], w_scale [N]")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x8.device)
    if out.shape != (M, N) or (bias is not None and bias.shape != (N,)):
        raise ValueError("out must be [M, N] and bias [N]")
    dt = out.dtype
    code = _code(dt)
    if not (_good(dev, torch.int8, x8, w8) and _good(dev, torch.float32, x_scale, w_scale) and _good(dev, dt, out)
            and (bias is None or _good(dev, dt, bias))):
        _refuse(x8=(x8, torch.int8), x_scale=(x_scale, torch.float32), w8=(w8, torch.int8),
                w_scale=(w_scale, torch.float32), out=(out, dt), **({} if bias is None else {"bias": (bias, dt)}))
    _check("oasr_linear_w8a8", L.oasr_linear_w8a8(
        x8.data_ptr(), x_scale.data_ptr(), w8.data_ptr(), w_scale.data_ptr(),
        None if bias is None else bias.data_ptr(), out.data_ptr(), M, N, K, code, _stream(stream)))
    return out


def oasr_project_qkv_pos_w8a8(x8, x_scale, w_qkv8, w_qkv_scale, b_qkv, pos8, pos_scale, w_pos8,
                              w_pos_scale, H, q=None, k=None, v=None, rel=None, stream=None):
    """q, k, v [M,H,64] and rel [R,H,64] by 8-bit integer products, one launch; the outputs have
    b_qkv's dtype.  Returns (q, k, v, rel)."""
    L, dev = _lib_device()
    M, d = x8.shape
    R = pos8.shape[0]
    _fits(M, R, d)
    if w_qkv8.shape != (3 * d, d) or w_qkv_scale.shape != (3 * d,) or b_qkv.shape != (3 * d,) or \
            pos8.shape != (R, d) or w_pos8.shape != (d, d) or w_pos_scale.shape != (d,) or \
            x_scale.shape != (M,) or pos_scale.shape != (R,) or d % H:
        raise ValueError("shapes: x8 [M,d], x_scale [M], w_qkv8 [3d,d], w_qkv_scale and b_qkv [3d], "
                         "pos8 [R,d], pos_scale [R], w_pos8 [d,d], w_pos_scale [d]")
    D, dt = d // H, b_qkv.dtype
    code = _code(dt)
    rows = (M, H, D)
    device = x8.device
    if q is None:
        q = torch.empty(rows, dtype=dt, device=device)
    if k is None:
        k = torch.empty_like(q)
    if v is None:
        v = torch.empty_like(q)
    if rel is None:
        rel = torch.empty((R, H, D), dtype=dt, device=device)
    if q.shape != rows or k.shape != rows or v.shape != rows or rel.shape != (R, H, D):
        raise ValueError("q, k, v must be [M, H, d/H] and rel [R, H, d/H]")
    i8, f32 = torch.int8, torch.float32
    if not (_good(dev, i8, x8, w_qkv8, pos8, w_pos8) and _good(dev, dt, b_qkv, q, k, v, rel)
            and _good(dev, f32, x_scale, w_qkv_scale, pos_scale, w_pos_scale)):
        _refuse(x8=(x8, i8), x_scale=(x_scale, f32), w_qkv8=(w_qkv8, i8), w_qkv_scale=(w_qkv_scale, f32),
                b_qkv=(b_qkv, dt), pos8=(pos8, i8), pos_scale=(pos_scale, f32), w_pos8=(w_pos8, i8),
                w_pos_scale=(w_pos_scale, f32), q=(q, dt), k=(k, dt), v=(v, dt), rel=(rel, dt))
    _check("oasr_project_qkv_pos_w8a8", L.oasr_project_qkv_pos_w8a8(
        x8.data_ptr(), x_scale.data_ptr(), w_qkv8.data_ptr(), w_qkv_scale.data_ptr(), b_qkv.data_ptr(),
        pos8.data_ptr(), pos_scale.data_ptr(), w_pos8.data_ptr(), w_pos_scale.data_ptr(), q.data_ptr(), k.data_ptr(),
        v.data_ptr(), rel.data_ptr(), M, R, d, H, code, _stream(stream)))
    return q, k, v, rel


def _rows_apart(t, name, dtype, dev) -> int:
    """Values from row to row of t [rows, H, D], whose rows are contiguous each but may lie apart (half of a
    product's columns); 16-byte steps."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or dev < 0 or t.dtype is not dtype:
        _dev(t, name, dtype)
    n, H, D = t.shape
    if n <= 1 or t.is_contiguous():
        if n == 1 and not t[0].is_contiguous():
            raise ValueError(f"{name} must have contiguous rows")
        return H * D
    apart, head, one = t.stride()
    if (one != 1 and D > 1) or (head != D and H > 1):
        raise ValueError(f"{name} must have contiguous rows")
    if apart < H * D or apart * t.element_size() % 16:
        raise ValueError(f"{name}'s rows must lie a multiple of 16 bytes apart and not overlap")
    return apart


def oasr_block_table_update(block_table, cache_seqlens, new_seqlens, free_blocks, free_state, block_size, total,
                            slot_map=None, cu_seqlens=None, stream=None):
    """Pages for streams that change from cache_seqlens to new_seqlens frames (int32 [B] each), taken
    from and given back to the ring of free block ids (free_blocks int32 [num_blocks], free_state int32
    [4]: first place, count, pages short, 0), in place.  Returns (slot_map int32 [total], the pool row
    of every new frame, stream after stream, -1 behind the last and where the ring was short; cu_seqlens
    int32 [B + 1], the streams' offsets in it).  Where it was short (free_state[2] > 0) no stream has grown, and
    only the shorter lengths are committed.  Entries of the table without a page are -1."""
    L, dev = _lib_device()
    table = block_table.shape
    total, block_size = int(total), int(block_size)
    if len(table) != 2 or cache_seqlens.shape != (table[0],) or new_seqlens.shape != (table[0],):
        raise ValueError("block_table must be [B, mbps], cache_seqlens and new_seqlens [B]")
    if free_blocks.dim() != 1 or free_state.shape != (4,):
        raise ValueError("free_blocks must be [num_blocks] and free_state [4]")
    _fits(table[0], table[1], total, block_size, free_blocks.shape[0])
    if total < 0:
        raise ValueError("total must not be negative")
    if slot_map is None:
        slot_map = block_table.new_empty((total,))
    if cu_seqlens is None:
        cu_seqlens = block_table.new_empty((table[0] + 1,))
    if slot_map.shape != (total,) or cu_seqlens.shape != (table[0] + 1,):
        raise ValueError("slot_map must be [total] and cu_seqlens [B + 1]")
    i32 = torch.int32
    if not _good(dev, i32, block_table, cache_seqlens, new_seqlens, free_blocks, free_state, slot_map, cu_seqlens):
        _refuse(block_table=(block_table, i32), cache_seqlens=(cache_seqlens, i32), new_seqlens=(new_seqlens, i32),
                free_blocks=(free_blocks, i32), free_state=(free_state, i32), slot_map=(slot_map, i32),
                cu_seqlens=(cu_seqlens, i32))
    _check("oasr_block_table_update", L.oasr_block_table_update(
        block_table.data_ptr(), cache_seqlens.data_ptr(), new_seqlens.data_ptr(), table[0], table[1], block_size,
        free_blocks.data_ptr(), free_blocks.shape[0], free_state.data_ptr(), slot_map.data_ptr(), total,
        cu_seqlens.data_ptr(), _stream(stream)))
    return slot_map, cu_seqlens


def oasr_paged_append_slots(k_new, v_new, k_pool, v_pool, slot_map, stream=None):
    """Write row i of k_new and v_new ([total,H,D], rows may lie apart) into row slot_map[i] of the pools
    ([nb,bs,H,D] as rows), in place; slots of -1 are skipped.  No rows (a step in which streams only end):
    nothing to do, here and in the calls below."""
    L, dev = _lib_device()
    dt = k_new.dtype
    code = _code(dt)
    n, H, D = k_new.shape
    if v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must share their shape [total, H, D]")
    shape = k_pool.shape
    if len(shape) != 4 or shape[2] != H or shape[3] != D or v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must be [num_blocks, block_size, H, D]")
    if slot_map.shape != (n,):
        raise ValueError("slot_map must be [total]")
    _fits(n, H, D, shape[0], shape[1])
    k_apart, v_apart = _rows_apart(k_new, "k_new", dt, dev), _rows_apart(v_new, "v_new", dt, dev)
    if not (_good(dev, dt, k_pool, v_pool) and _good(dev, torch.int32, slot_map)):
        _refuse(k_pool=(k_pool, dt), v_pool=(v_pool, dt), slot_map=(slot_map, torch.int32))
    if n == 0:
        return
    _check("oasr_paged_append_slots", L.oasr_paged_append_slots(
        k_new.data_ptr(), v_new.data_ptr(), k_apart, v_apart, k_pool.data_ptr(), v_pool.data_ptr(), shape[0], shape[1],
        slot_map.data_ptr(), n, H, D, code, _stream(stream)))


def _cross(dev, q, cu_q, max_q, Hkv, out):
    """Checks what both forms of the cross attention take; returns the output, total_q, N, H, D, q's
    row stride and the dtype's code."""
    dt = q.dtype
    code = _code(dt)
    n, H, D = q.shape
    if Hkv < 1 or H % Hkv:
        raise ValueError("q's heads must be a multiple of k's")
    if cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError("cu_q must be [num_seqs + 1]")
    _fits(n, H, D, cu_q.shape[0], max_q)
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty((n, H, D))
    elif out.shape != (n, H, D):
        raise ValueError("out must be [total_q, H, D]")
    apart = _rows_apart(q, "q", dt, dev)
    if not (_good(dev, dt, out) and _good(dev, torch.int32, cu_q)):
        _refuse(out=(out, dt), cu_q=(cu_q, torch.int32))
    return out, n, cu_q.shape[0] - 1, H, D, apart, code


def oasr_cross_attn_packed(q, k, v, cu_q, cu_k, max_q, max_k, out=None, scale=None, stream=None):
    """Cross attention of packed queries [total_q,H,64] (sequence s: rows cu_q[s] to cu_q[s+1]) over packed
    keys and values [total_k,Hkv,64] (cu_k), Hkv dividing H; rows of q, k and v may lie apart.  max_q and
    max_k: the longest sequences' lengths.  Returns out [total_q,H,64]; without keys zeros (k and v have a
    row all the same)."""
    L, dev = _lib_device()
    nk, Hkv, Dk = k.shape
    max_q, max_k = int(max_q), int(max_k)
    if v.shape != k.shape or Dk != q.shape[2]:
        raise ValueError("k and v must be [total_k, Hkv, D]")
    out, n, N, H, D, q_apart, code = _cross(dev, q, cu_q, max_q, Hkv, out)
    if cu_k.shape != cu_q.shape:
        raise ValueError("cu_k must have cu_q's length")
    _fits(nk, max_k)
    k_apart, v_apart = _rows_apart(k, "k", q.dtype, dev), _rows_apart(v, "v", q.dtype, dev)
    if not _good(dev, torch.int32, cu_k):
        _refuse(cu_k=(cu_k, torch.int32))
    if n == 0:
        return out
    _check("oasr_cross_attn_packed", L.oasr_cross_attn_packed(
        q.data_ptr(), q_apart, k.data_ptr(), k_apart, v.data_ptr(), v_apart, cu_q.data_ptr(), cu_k.data_ptr(), N, max_q,
        max_k, n, nk, out.data_ptr(), H, Hkv, D, D ** -0.5 if scale is None else scale, code, _stream(stream)))
    return out


def oasr_cross_attn_paged(q, k_pool, v_pool, block_table, cache_seqlens, cu_q, max_q, max_k=None, out=None, scale=None,
                          stream=None):
    """The same over keys and values in pages: the first cache_seqlens[s] positions of block_table[s] in the
    pools [nb,bs,Hkv,64].  max_k: the longest sequence's keys (None: the table's width)."""
    L, dev = _lib_device()
    shape, table = k_pool.shape, block_table.shape
    if len(shape) != 4 or shape[3] != q.shape[2]:
        raise ValueError("k_pool must be [num_blocks, block_size, Hkv, D]")
    if v_pool.shape != shape:
        raise ValueError("v_pool must have k_pool's shape")
    if len(table) != 2 or cu_q.shape != (table[0] + 1,) or cache_seqlens.shape != table[:1]:
        raise ValueError("block_table must be [num_seqs, mbps], cache_seqlens [num_seqs] and cu_q [num_seqs + 1]")
    max_q = int(max_q)
    out, n, N, H, D, q_apart, code = _cross(dev, q, cu_q, max_q, shape[2], out)
    max_k = table[1] * shape[1] if max_k is None else int(max_k)
    _fits(shape[0], shape[1], table[1], max_k)
    if not (_good(dev, q.dtype, k_pool, v_pool) and _good(dev, torch.int32, block_table, cache_seqlens)):
        _refuse(k_pool=(k_pool, q.dtype), v_pool=(v_pool, q.dtype), block_table=(block_table, torch.int32),
                cache_seqlens=(cache_seqlens, torch.int32))
    if n == 0:
        return out
    _check("oasr_cross_attn_paged", L.oasr_cross_attn_paged(
        q.data_ptr(), q_apart, k_pool.data_ptr(), v_pool.data_ptr(), shape[0], shape[1], block_table.data_ptr(), table[1],
        cache_seqlens.data_ptr(), cu_q.data_ptr(), N, max_q, max_k, n, out.data_ptr(), H, shape[2], D,
        D ** -0.5 if scale is None else scale, code, _stream(stream)))
    return out


def _blocks(x8, scale, name):
    """Rows, row length and blocks of a matrix held in blocks of 128."""
    M, K = x8.shape
    if scale.shape != (M, -(-K // 128)):
        raise ValueError(f"{name}'s scale must be [rows, ceil(K / 128)]")
    return M, K


def oasr_quantize_blocks(x, x8=None, scale=None, stream=None):
    """Rows of x [M,K] in e4m3 with one power-of-two scale for each 128 values; returns (x8 float8_e4m3fn
    [M,K], scale uint8 [M, ceil(K/128)], the byte e + 127 standing for 2^e)."""
    L, dev = _lib_device()
    dt = x.dtype
    code = _code(dt)
    M, K = x.shape
    _fits(M, K)
    if x8 is None:
        x8 = torch.empty_like(x, dtype=torch.float8_e4m3fn)   # x is contiguous, or refused below
    if scale is None:
        scale = x.new_empty((M, -(-K // 128)), dtype=torch.uint8)
    if x8.shape != (M, K):
        raise ValueError("x8 must be [M, K]")
    _blocks(x8, scale, "x8")
    if not (_good(dev, dt, x) and _good(dev, torch.float8_e4m3fn, x8) and _good(dev, torch.uint8, scale)):
        _refuse(x=(x, dt), x8=(x8, torch.float8_e4m3fn), scale=(scale, torch.uint8))
    if M == 0:
        return x8, scale
    _check("oasr_quantize_blocks", L.oasr_quantize_blocks(
        x.data_ptr(), x8.data_ptr(), scale.data_ptr(), M, K, code, _stream(stream)))
    return x8, scale


def oasr_linear_e4m3(x8, x_scale, w8, w_scale, bias=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """x . w^T + bias of rows held as `oasr_quantize_blocks` leaves them (x8 [M,K], w8 [N,K]); returns out
    [M,N] of ``out_dtype`` (or of the out given)."""
    L, dev = _lib_device()
    M, K = _blocks(x8, x_scale, "x8")
    N, Kw = _blocks(w8, w_scale, "w8")
    _fits(M, N, K)
    if Kw != K:
        raise ValueError("shapes: x8 [M,K], w8 [N,K]")
    if out is None:
        out = x8.new_empty((M, N), dtype=out_dtype)
    if out.shape != (M, N) or (bias is not None and bias.shape != (N,)):
        raise ValueError("out must be [M, N] and bias [N]")
    dt = out.dtype
    code = _code(dt)
    e4 = torch.float8_e4m3fn
    if not (_good(dev, e4, x8, w8) and _good(dev, torch.uint8, x_scale, w_scale) and _good(dev, dt, out)
            and (bias is None or _good(dev, dt, bias))):
        _refuse(x8=(x8, e4), x_scale=(x_scale, torch.uint8), w8=(w8, e4), w_scale=(w_scale, torch.uint8), out=(out, dt),
                **({} if bias is None else {"bias": (bias, dt)}))
    if M == 0:
        return out
    _check("oasr_linear_e4m3", L.oasr_linear_e4m3(
        x8.data_ptr(), x_scale.data_ptr(), w8.data_ptr(), w_scale.data_ptr(), None if bias is None else bias.data_ptr(),
        out.data_ptr(), M, N, K, code, _stream(stream)))
    return out


def oasr_device_status(clear: bool = True) -> int:
    """Raw device status bits (1 = an index was out of range, 2 = a wait timed out)."""
    L = load()
    flags = ctypes.c_uint(0)
    _check("oasr_device_status", L.oasr_device_status(ctypes.byref(flags), int(clear)))
    return int(flags.value)


def oasr_version() -> int:
    return int(load().oasr_version())


def oasr_selftest_wait(limit_us: int = 20000, stream=None) -> None:
    """Diagnostic: the library's bounded wait on a barrier that nothing signals.  It runs
    out after ``limit_us`` microseconds and raises the timeout bit (2) of the device status
    word, as any of the library's kernels does when a copy it waits for never lands."""
    _check("oasr_selftest_wait", load().oasr_selftest_wait(int(limit_us), _stream(stream)))


# NVTX ranges around every call into the library, for Nsight timelines: set OASR_NVTX=1
# before the import.
NVTX = os.environ.get("OASR_NVTX", "") == "1"


def _traced(fn):
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        torch.cuda.nvtx.range_push(fn.__name__)
        try:
            return fn(*args, **kwargs)
        finally:
            torch.cuda.nvtx.range_pop()
    return wrapper


if NVTX:
    for _name in ("oasr_paged_append", "oasr_chunk_relattn_paged", "oasr_chunk_step_paged",
                  "oasr_packed_relattn_varlen", "oasr_packed_relattn_chunked", "oasr_window_commit",
                  "oasr_project_qkv_pos", "oasr_selftest_wait", "oasr_paged_append_e4m3",
                  "oasr_paged_read_e4m3", "oasr_chunk_relattn_paged_e4m3",
                  "oasr_chunk_step_paged_e4m3", "oasr_quantize_rows", "oasr_linear_w8a8",
                  "oasr_project_qkv_pos_w8a8", "oasr_block_table_update", "oasr_paged_append_slots",
                  "oasr_cross_attn_packed", "oasr_cross_attn_paged", "oasr_quantize_blocks",
                  "oasr_linear_e4m3"):
        globals()[_name] = _traced(globals()[_name])
