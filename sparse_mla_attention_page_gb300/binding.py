"""Thin ctypes binding of the C ABI in include/dsa.h (argument marshalling only).

Every function here has the name of the C entry point it calls, takes torch
tensors that already live on the GPU, checks that they have the dtype and
shape the C function documents, passes their pointers and sizes, and turns a
non-zero status into ``DsaError``.  All computation happens in the CUDA
library; there is no fallback: if ``libdsa_gb300.so`` has not been built the
first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

DSA_KV_RAW512 = 0
DSA_KV_SCALED528 = 1
DSA_KV_ROPE656 = 2
DSA_KV_FP4_288 = 16
DSA_KV_FP4_416 = 17
LAYOUTS = {"raw512": DSA_KV_RAW512, "scaled528": DSA_KV_SCALED528, "rope656": DSA_KV_ROPE656,
           "fp4_288": DSA_KV_FP4_288, "fp4_416": DSA_KV_FP4_416}
_ROW_BYTES = {DSA_KV_RAW512: 512, DSA_KV_SCALED528: 528, DSA_KV_ROPE656: 656, DSA_KV_FP4_288: 288, DSA_KV_FP4_416: 416}

DSA_DEV_ERR_INDEX_RANGE = 1
DSA_DEV_ERR_PAGE_RANGE = 2
DSA_DEV_ERR_TIMEOUT = 4
DSA_DEV_ERR_SLOT_RANGE = 8
DSA_DEV_ERR_LENGTH = 16
DSA_DEV_ERR_NO_PAGES = 32

_lock = threading.Lock()
_lib = None

# Every symbol include/dsa.h declares.
EXPORTS = (
    "dsa_status_string", "dsa_kv_row_bytes", "dsa_kv_write_raw", "dsa_kv_write_scaled", "dsa_kv_write_rope656",
    "dsa_quantize_q8", "dsa_sparse_attn_workspace_bytes", "dsa_sparse_attn_decode",
    "dsa_sparse_attn_prefill_q8", "dsa_gather_dequant_workspace_bytes", "dsa_gather_dequant",
    "dsa_sparse_attn_decode_noalloc", "dsa_set_wait_limit_ns",
    "dsa_pages_extend", "dsa_pages_release", "dsa_rope_qkv656", "dsa_chunk_attn_workspace_bytes", "dsa_chunk_attn",
    "dsa_kv_write_fp4", "dsa_kv_read", "dsa_pages_release_own", "dsa_prefix_attn_workspace_bytes", "dsa_prefix_attn",
)


class DsaRope(ctypes.Structure):
    """dsa_rope of include/dsa.h; ``rope_spec`` fills one."""
    _fields_ = [("inv_freq", ctypes.c_double * 32), ("axis", ctypes.c_int32 * 32), ("n_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float)]


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build the CUDA library first "
                                   "(sparse_mla_attention_page_gb300.build.build())")
            L = ctypes.CDLL(path)
            c = ctypes
            vp, i64, i32 = c.c_void_p, c.c_int64, c.c_int
            L.dsa_status_string.restype = c.c_char_p
            L.dsa_status_string.argtypes = [i32]
            L.dsa_set_wait_limit_ns.restype = c.c_uint64
            L.dsa_set_wait_limit_ns.argtypes = [c.c_uint64]
            L.dsa_kv_row_bytes.restype = c.c_size_t
            L.dsa_kv_row_bytes.argtypes = [i32]
            for f in (L.dsa_kv_write_raw, L.dsa_kv_write_scaled, L.dsa_kv_write_rope656):
                f.restype = i32
                f.argtypes = [vp, i64, vp, vp, i64, vp, vp]
            L.dsa_quantize_q8.restype = i32
            L.dsa_quantize_q8.argtypes = [vp, i64, vp, vp, vp]
            L.dsa_sparse_attn_workspace_bytes.restype = c.c_size_t
            L.dsa_sparse_attn_workspace_bytes.argtypes = [i32, i32, i32]
            L.dsa_sparse_attn_decode.restype = i32
            L.dsa_sparse_attn_decode.argtypes = [
                vp, i32, i32, i32, vp, i64, i32, i32, vp, i32, i32, i32, vp, vp, i32,
                c.c_float, vp, vp, vp, c.c_size_t, vp, vp]
            L.dsa_sparse_attn_prefill_q8.restype = i32
            L.dsa_sparse_attn_prefill_q8.argtypes = [
                vp, vp, i32, i32, i32, vp, i64, i32, i32, vp, i32, i32, i32, vp, vp, i32,
                c.c_float, vp, vp, vp, c.c_size_t, vp, vp]
            L.dsa_gather_dequant.restype = i32
            L.dsa_gather_dequant.argtypes = [vp, i64, i32, vp, i32, i32, i32, vp, vp, i32, i32, vp, c.c_size_t,
                                             vp, vp, vp]
            L.dsa_gather_dequant_workspace_bytes.restype = c.c_size_t
            L.dsa_gather_dequant_workspace_bytes.argtypes = [i32, i32, i64, i32]
            L.dsa_sparse_attn_decode_noalloc.restype = i32
            L.dsa_sparse_attn_decode_noalloc.argtypes = [
                vp, i32, i32, i32, vp, i64, i32, i32, vp, i32, i32, i32, vp, vp, i32,
                c.c_float, vp, vp, vp, vp]
            L.dsa_pages_extend.restype = i32
            L.dsa_pages_extend.argtypes = [vp, vp, i32, vp, i32, i32, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp]
            L.dsa_pages_release.restype = i32
            L.dsa_pages_release.argtypes = [vp, vp, i32, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp]
            L.dsa_rope_qkv656.restype = i32
            L.dsa_rope_qkv656.argtypes = [c.POINTER(DsaRope), vp, i64, i32, i32, vp, i64, i64, vp, i64, i64, vp,
                                          vp, i64, vp, i64, vp, vp, i64, vp, vp]
            L.dsa_chunk_attn_workspace_bytes.restype = c.c_size_t
            L.dsa_chunk_attn_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.dsa_chunk_attn.restype = i32
            L.dsa_chunk_attn.argtypes = [vp, i32, i32, i32, vp, i64, i32, i32, vp, i32, i32, i32, vp, vp, i32,
                                         c.c_float, vp, vp, vp, c.c_size_t, vp, vp]
            L.dsa_kv_write_fp4.restype = i32
            L.dsa_kv_write_fp4.argtypes = [vp, i64, vp, i64, i64, vp, vp, i64, vp, vp]
            L.dsa_kv_read.restype = i32
            L.dsa_kv_read.argtypes = [vp, i64, i32, vp, i32, i32, i32, vp, vp, vp, i64, i64, vp, vp]
            L.dsa_pages_release_own.restype = i32
            L.dsa_pages_release_own.argtypes = [vp, vp, vp, i32, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp]
            L.dsa_prefix_attn_workspace_bytes.restype = c.c_size_t
            L.dsa_prefix_attn_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.dsa_prefix_attn.restype = i32
            L.dsa_prefix_attn.argtypes = [vp, i32, i32, i32, vp, i64, i32, i32, vp, i32, i32, i32, vp, vp, vp, vp, i32, i32,
                                          c.c_float, vp, vp, vp, c.c_size_t, vp, vp]
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().dsa_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise DsaError(status, where)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, last: int | None = None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if last is not None and t.shape[-1] != last:
        raise ValueError(f"{name} must have last dimension {last}, got {tuple(t.shape)}")


def dsa_set_wait_limit_ns(ns: int) -> int:
    """Limit of the attention kernel's bounded waits for later calls; returns the old one."""
    return int(lib().dsa_set_wait_limit_ns(int(ns)))


def dsa_kv_row_bytes(layout) -> int:
    return int(lib().dsa_kv_row_bytes(LAYOUTS.get(layout, layout)))


def _write(fn_name, x_bf16, slots, pool, err_flag, stream, width=512):
    _need(x_bf16, "x_bf16", torch.bfloat16, width)
    _need(slots, "slots", torch.int64)
    _need(pool, "pool", torch.uint8)
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    n = x_bf16.numel() // width
    if slots.numel() != n:
        raise ValueError("slots must have one entry per row")
    rows = pool.shape[0]
    st = getattr(lib(), fn_name)(_ptr(x_bf16), n, _ptr(slots), _ptr(pool), rows, _ptr(err_flag), _stream(stream))
    _check(st, fn_name)


def dsa_kv_write_raw(x_bf16, slots, pool, err_flag=None, stream=None) -> None:
    """pool [rows, 512] uint8 <- e4m3(x) at rows ``slots`` (see include/dsa.h)."""
    if pool.dim() != 2 or pool.shape[1] != 512:
        raise ValueError("raw pool must be [rows, 512] uint8")
    _write("dsa_kv_write_raw", x_bf16, slots, pool, err_flag, stream)


def dsa_kv_write_scaled(x_bf16, slots, pool, err_flag=None, stream=None) -> None:
    """pool [rows, 528] uint8 <- group-scaled e4m3(x) at rows ``slots``."""
    if pool.dim() != 2 or pool.shape[1] != 528:
        raise ValueError("scaled pool must be [rows, 528] uint8")
    _write("dsa_kv_write_scaled", x_bf16, slots, pool, err_flag, stream)


def dsa_kv_write_rope656(x_bf16, slots, pool, err_flag=None, stream=None) -> None:
    """pool [rows, 656] uint8 <- group-scaled e4m3(x[:, :512]) and the BF16 RoPE
    dims x[:, 512:576] at rows ``slots``."""
    if pool.dim() != 2 or pool.shape[1] != 656:
        raise ValueError("RoPE pool must be [rows, 656] uint8")
    _write("dsa_kv_write_rope656", x_bf16, slots, pool, err_flag, stream, width=576)


def dsa_quantize_q8(q_bf16, q8, q_scale, stream=None) -> None:
    """q8 [..., 512] uint8 and q_scale [...] float32 from q_bf16 [..., 512]."""
    _need(q_bf16, "q_bf16", torch.bfloat16, 512)
    _need(q8, "q8", torch.uint8, 512)
    _need(q_scale, "q_scale", torch.float32)
    n = q_bf16.numel() // 512
    if q8.numel() != n * 512 or q_scale.numel() != n:
        raise ValueError("q8 / q_scale sizes do not match q_bf16")
    _check(lib().dsa_quantize_q8(_ptr(q_bf16), n, _ptr(q8), _ptr(q_scale), _stream(stream)),
           "dsa_quantize_q8")


def dsa_sparse_attn_workspace_bytes(T: int, H: int, K: int) -> int:
    return int(lib().dsa_sparse_attn_workspace_bytes(int(T), int(H), int(K)))


def workspace_for(T: int, H: int, K: int, device=None) -> torch.Tensor | None:
    """A device workspace of the size the attention entry points need (or None)."""
    n = dsa_sparse_attn_workspace_bytes(T, H, K)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _attn_common(q, pool, layout, topk, o, lse, page_table, token_seq, workspace, err_flag):
    T, H = q.shape[0], q.shape[1]
    _need(pool, "pool", torch.uint8)
    _need(topk, "topk", torch.int32)
    _need(o, "o", torch.bfloat16, 512)
    _need(lse, "lse", torch.float32)
    if topk.dim() != 2 or topk.shape[0] != T:
        raise ValueError("topk must be [T, K] int32")
    if tuple(o.shape) != (T, H, 512) or tuple(lse.shape) != (T, H):
        raise ValueError("o must be [T, H, 512] bf16 and lse [T, H] float32")
    lay = LAYOUTS.get(layout, layout)
    if page_table is not None:
        _need(page_table, "page_table", torch.int32)
        B, max_pages = page_table.shape
    else:
        B, max_pages = 1, 1
    if token_seq is not None:
        _need(token_seq, "token_seq", torch.int32)
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return T, H, lay, B, max_pages, ws_bytes


def dsa_gather_dequant_workspace_bytes(T: int, K: int, pool_rows: int, layout) -> int:
    return int(lib().dsa_gather_dequant_workspace_bytes(T, K, pool_rows, LAYOUTS.get(layout, layout)))


def gather_workspace_for(T: int, K: int, pool_rows: int, layout, device=None) -> torch.Tensor:
    """A BF16 workspace [min(pool_rows, T*K), 512 or 576] for dsa_gather_dequant."""
    lay = LAYOUTS.get(layout, layout)
    width = 576 if lay == DSA_KV_ROPE656 else 512
    rows = min(pool_rows, T * K)
    return torch.empty(rows, width, dtype=torch.bfloat16, device=device or "cuda")


def dsa_gather_dequant(pool, layout, topk, out, idx_out, page_table=None, page_size=64,
                       token_seq=None, err_flag=None, stream=None) -> None:
    """BF16 workspace out [min(pool_rows, T*K), 512 or 576] and remapped indices
    idx_out [T, K] for topk [T, K]."""
    lay = LAYOUTS.get(layout, layout)
    _need(pool, "pool", torch.uint8)
    _need(topk, "topk", torch.int32)
    _need(out, "out", torch.bfloat16, 576 if lay == DSA_KV_ROPE656 else 512)
    _need(idx_out, "idx_out", torch.int32)
    if topk.dim() != 2:
        raise ValueError("topk must be [T, K] int32")
    T, K = topk.shape
    if tuple(idx_out.shape) != (T, K):
        raise ValueError("idx_out must be [T, K] int32")
    if page_table is not None:
        _need(page_table, "page_table", torch.int32)
        B, max_pages = page_table.shape
    else:
        B, max_pages = 1, 1
    if token_seq is not None:
        _need(token_seq, "token_seq", torch.int32)
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    _check(lib().dsa_gather_dequant(_ptr(pool), pool.shape[0], lay, _ptr(page_table), B, max_pages,
                                    page_size, _ptr(token_seq), _ptr(topk), T, K, _ptr(out),
                                    out.numel() * out.element_size(), _ptr(idx_out), _ptr(err_flag),
                                    _stream(stream)),
           "dsa_gather_dequant")


def _kv_row_dim(pool, lay) -> int:
    """Key width held by one pool row (528- and 656-byte rows carry 16 bytes of
    scales; 656-byte rows add 64 BF16 RoPE dims; 4-bit rows hold 512 dims in 288
    bytes): 512 or 576 for the layout's own row size alone."""
    if lay in (DSA_KV_FP4_288, DSA_KV_FP4_416):
        return pool.shape[1] + (224 if lay == DSA_KV_FP4_288 else 160)
    if lay == DSA_KV_ROPE656:
        return pool.shape[1] - 80
    return pool.shape[1] - (16 if lay == DSA_KV_SCALED528 else 0)


def dsa_sparse_attn_decode(q_bf16, pool, layout, topk, sm_scale, o, lse, workspace=None,
                           page_table=None, page_size=64, token_seq=None, err_flag=None,
                           stream=None) -> None:
    """Sparse MLA decode with BF16 queries [T, H, 512] ([T, H, 576] over 656-byte
    rows; see include/dsa.h)."""
    _need(q_bf16, "q_bf16", torch.bfloat16, 576 if LAYOUTS.get(layout, layout) == DSA_KV_ROPE656 else 512)
    T, H, lay, B, max_pages, ws_bytes = _attn_common(q_bf16, pool, layout, topk, o, lse,
                                                     page_table, token_seq, workspace, err_flag)
    st = lib().dsa_sparse_attn_decode(
        _ptr(q_bf16), T, H, q_bf16.shape[-1], _ptr(pool), pool.shape[0], lay,
        _kv_row_dim(pool, lay),
        _ptr(page_table), B, max_pages, page_size, _ptr(token_seq), _ptr(topk), topk.shape[1],
        float(sm_scale), _ptr(o), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(err_flag),
        _stream(stream))
    _check(st, "dsa_sparse_attn_decode")


def dsa_sparse_attn_prefill_q8(q8, q_scale, pool, layout, topk, sm_scale, o, lse, workspace=None,
                               page_table=None, page_size=64, token_seq=None, err_flag=None,
                               stream=None) -> None:
    """Sparse MLA prefill with E4M3 queries [T, H, 512] + FP32 scales [T, H]."""
    _need(q8, "q8", torch.uint8, 512)
    _need(q_scale, "q_scale", torch.float32)
    T, H, lay, B, max_pages, ws_bytes = _attn_common(q8, pool, layout, topk, o, lse,
                                                     page_table, token_seq, workspace, err_flag)
    st = lib().dsa_sparse_attn_prefill_q8(
        _ptr(q8), _ptr(q_scale), T, H, q8.shape[-1], _ptr(pool), pool.shape[0], lay,
        _kv_row_dim(pool, lay),
        _ptr(page_table), B, max_pages, page_size, _ptr(token_seq), _ptr(topk), topk.shape[1],
        float(sm_scale), _ptr(o), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(err_flag),
        _stream(stream))
    _check(st, "dsa_sparse_attn_prefill_q8")


def dsa_sparse_attn_decode_noalloc(q_bf16, pool, layout, topk, sm_scale, o, lse, page_table=None,
                                   page_size=64, token_seq=None, err_flag=None, stream=None) -> None:
    """Decode using the library's own static workspace (no allocation by anyone);
    see include/dsa.h for its size limit and the sharing rules."""
    _need(q_bf16, "q_bf16", torch.bfloat16, 576 if LAYOUTS.get(layout, layout) == DSA_KV_ROPE656 else 512)
    T, H, lay, B, max_pages, _ = _attn_common(q_bf16, pool, layout, topk, o, lse,
                                              page_table, token_seq, None, err_flag)
    st = lib().dsa_sparse_attn_decode_noalloc(
        _ptr(q_bf16), T, H, q_bf16.shape[-1], _ptr(pool), pool.shape[0], lay, _kv_row_dim(pool, lay),
        _ptr(page_table), B, max_pages, page_size, _ptr(token_seq), _ptr(topk), topk.shape[1],
        float(sm_scale), _ptr(o), _ptr(lse), _ptr(err_flag), _stream(stream))
    _check(st, "dsa_sparse_attn_decode_noalloc")


# ------------------------------------------------ dense serving operators

def _refuse(t, name, dtype, shape, device, strided):
    """Raises what is wrong with an argument that _arg turned down."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's device is cuda:{device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if strided:
        raise ValueError(f"{name} must be contiguous in its last dim")
    raise TypeError(f"{name} must be contiguous")


def _arg(t, name: str, dtype: torch.dtype, shape, device: int):
    """Address of a contiguous tensor of the given type and shape (None: any) on the call's device."""
    try:
        if t.dtype is dtype and t.get_device() == device and (shape is None or t.shape == shape) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:       # not a tensor
        pass
    _refuse(t, name, dtype, shape, device, False)


def _arg_strided(t, name: str, dtype: torch.dtype, shape, device: int):
    """The same for a tensor that is contiguous in its last dim only; None stays None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == device and t.shape == shape and (t.stride(-1) == 1 or t.shape[-1] == 1):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, device, True)


def _flag(t, device: int):
    return None if t is None else _arg(t, "err_flag", torch.int32, None, device)


def _dims(t, name: str, n: int):
    """The shape of a tensor of n dims."""
    s = getattr(t, "shape", ())
    if len(s) != n:
        raise ValueError(f"{name} must be a tensor of {n} dims")
    return s


def _call_device(stream):
    """(the current device, the stream's address on it)."""
    dev = torch._C._cuda_getDevice()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def dsa_pages_extend(seq_lens, new_lens, page_table, page_size, free_pages, free_count, free_count_out, slots,
                     positions, token_seq, cu_q, kv_lens, err_flag=None, stream=None) -> None:
    """Pages for new_lens [B] more tokens of requests that hold seq_lens [B], off the stack
    free_pages[:free_count], into page_table [B, max_pages]; and the step's token rows: slots (int64),
    positions and token_seq [T], cu_q [B + 1] and kv_lens [B] (see include/dsa.h).  free_count_out may be
    free_count, kv_lens may be seq_lens."""
    dev, s = _call_device(stream)
    i32 = torch.int32
    B, W = _dims(page_table, "page_table", 2)
    T, = _dims(slots, "slots", 1)
    cap, = _dims(free_pages, "free_pages", 1)
    _check((_lib or lib()).dsa_pages_extend(
        _arg(seq_lens, "seq_lens", i32, (B,), dev), _arg(new_lens, "new_lens", i32, (B,), dev), B,
        _arg(page_table, "page_table", i32, None, dev), W, page_size, _arg(free_pages, "free_pages", i32, None, dev), cap,
        _arg(free_count, "free_count", i32, (1,), dev), _arg(free_count_out, "free_count_out", i32, (1,), dev), T,
        _arg(slots, "slots", torch.int64, None, dev), _arg(positions, "positions", i32, (T,), dev),
        _arg(token_seq, "token_seq", i32, (T,), dev), _arg(cu_q, "cu_q", i32, (B + 1,), dev),
        _arg(kv_lens, "kv_lens", i32, (B,), dev), _flag(err_flag, dev), s), "dsa_pages_extend")


def dsa_pages_release(finished, seq_lens, page_table, page_size, free_pages, free_count, free_count_out, seq_lens_out,
                      err_flag=None, stream=None) -> None:
    """Pushes the pages of the finished requests (bool [B]) onto the stack free_pages[:free_count] (see
    include/dsa.h).  free_count_out may be free_count, seq_lens_out may be seq_lens."""
    dev, s = _call_device(stream)
    i32 = torch.int32
    B, W = _dims(page_table, "page_table", 2)
    cap, = _dims(free_pages, "free_pages", 1)
    _check((_lib or lib()).dsa_pages_release(
        _arg(finished, "finished", torch.bool, (B,), dev), _arg(seq_lens, "seq_lens", i32, (B,), dev), B,
        _arg(page_table, "page_table", i32, None, dev), W, page_size, _arg(free_pages, "free_pages", i32, None, dev), cap,
        _arg(free_count, "free_count", i32, (1,), dev), _arg(free_count_out, "free_count_out", i32, (1,), dev),
        _arg(seq_lens_out, "seq_lens_out", i32, (B,), dev), _flag(err_flag, dev), s), "dsa_pages_release")


def dsa_pages_release_own(finished, shared_pages, seq_lens, page_table, page_size, free_pages, free_count,
                          free_count_out, seq_lens_out, err_flag=None, stream=None) -> None:
    """dsa_pages_release, but for the first shared_pages [B] pages of each request, which belong to a prefix that
    other requests hold too (see include/dsa.h)."""
    dev, s = _call_device(stream)
    i32 = torch.int32
    B, W = _dims(page_table, "page_table", 2)
    cap, = _dims(free_pages, "free_pages", 1)
    _check((_lib or lib()).dsa_pages_release_own(
        _arg(finished, "finished", torch.bool, (B,), dev), _arg(shared_pages, "shared_pages", i32, (B,), dev),
        _arg(seq_lens, "seq_lens", i32, (B,), dev), B,
        _arg(page_table, "page_table", i32, None, dev), W, page_size, _arg(free_pages, "free_pages", i32, None, dev), cap,
        _arg(free_count, "free_count", i32, (1,), dev), _arg(free_count_out, "free_count_out", i32, (1,), dev),
        _arg(seq_lens_out, "seq_lens_out", i32, (B,), dev), _flag(err_flag, dev), s), "dsa_pages_release_own")


def dsa_kv_write_fp4(kv_c, slots, pool, k_pe=None, err_flag=None, stream=None) -> None:
    """pool [rows, 288] uint8 <- the latents kv_c [n, 512] in 4 bits at rows ``slots``; with k_pe [n, 64], pool
    [rows, 416] and the RoPE dims behind them (see include/dsa.h)."""
    dev, s = _call_device(stream)
    bf = torch.bfloat16
    n, _ = _dims(kv_c, "kv_c", 2)
    rows, _ = _dims(pool, "pool", 2)
    st = (lambda t: 0 if t is None or n <= 1 else t.stride(0))
    _check((_lib or lib()).dsa_kv_write_fp4(
        _arg_strided(kv_c, "kv_c", bf, (n, 512), dev), st(kv_c), _arg_strided(k_pe, "k_pe", bf, (n, 64), dev), st(k_pe), n,
        _arg(slots, "slots", torch.int64, (n,), dev),
        _arg(pool, "pool", torch.uint8, (rows, 288 if k_pe is None else 416), dev), rows, _flag(err_flag, dev), s),
        "dsa_kv_write_fp4")


def dsa_kv_read(pool, layout, page_table, page_size, cu_rows, out, starts=None, err_flag=None, stream=None) -> None:
    """out [n, 512 or 576] BF16 <- the rows of the requests in token order: request b's rows starts[b] (0) and on go to
    out[cu_rows[b]:cu_rows[b + 1]] (see include/dsa.h).  out may be strided in its first dim."""
    dev, s = _call_device(stream)
    lay = LAYOUTS.get(layout, layout)
    i32 = torch.int32
    B, W = _dims(page_table, "page_table", 2)
    rows, _ = _dims(pool, "pool", 2)
    n, _ = _dims(out, "out", 2)
    width = 576 if lay in (DSA_KV_ROPE656, DSA_KV_FP4_416) else 512
    _check((_lib or lib()).dsa_kv_read(
        _arg(pool, "pool", torch.uint8, (rows, _ROW_BYTES.get(lay)), dev), rows, lay,
        _arg(page_table, "page_table", i32, None, dev), B, W, page_size, _arg(cu_rows, "cu_rows", i32, (B + 1,), dev),
        None if starts is None else _arg(starts, "starts", i32, (B,), dev),
        _arg_strided(out, "out", torch.bfloat16, (n, width), dev), n, out.stride(0) if n > 1 else width,
        _flag(err_flag, dev), s), "dsa_kv_read")


def rope_spec(theta=10000.0, sections=(32,), interleaved=False, inv_freq=None, axis=None, mscale=1.0) -> DsaRope:
    """The rotary embedding of the 64 RoPE dims: pair i turns by positions[axis[i]] * inv_freq[i] radians.
    ``sections`` gives the first sections[0] pairs axis 0, the next sections[1] axis 1, ...; ``axis`` (32
    entries) sets any other assignment.  ``inv_freq`` (32 entries) replaces theta^(-i / 32)."""
    if axis is None:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    axis = [int(a) for a in axis]
    inv_freq = [float(theta) ** (-i / 32.0) for i in range(32)] if inv_freq is None else [float(f) for f in inv_freq]
    if len(axis) != 32 or len(inv_freq) != 32:
        raise ValueError("a rotary spec has 32 pairs: sections sum to 32, axis and inv_freq have 32 entries")
    return DsaRope((ctypes.c_double * 32)(*inv_freq), (ctypes.c_int32 * 32)(*axis), max(max(axis) + 1, len(sections)),
                   int(bool(interleaved)), mscale)


def dsa_rope_qkv656(q_nope, q_pe, q_out, kv_c, k_pe, slots, pool, positions, rope, err_flag=None, stream=None) -> None:
    """q_out [T, H, 576] <- q_nope [T, H, 512] and the turned q_pe [T, H, 64]; pool [rows, 656] <- the rows of
    kv_c [T, 512] and the turned k_pe [T, 64] at ``slots``; positions int32 [axes, T] (see include/dsa.h).
    q_nope None leaves q_out's latent part; q_pe and q_out None, or kv_c, k_pe, slots and pool None, leave that
    side out."""
    dev, s = _call_device(stream)
    bf = torch.bfloat16
    if q_pe is not None:
        T, H, _ = _dims(q_pe, "q_pe", 3)
    else:
        (T, _), H = _dims(kv_c, "kv_c", 2), 1
    st = (lambda t, d: 0 if t is None or t.shape[d] == 1 else t.stride(d))
    _check((_lib or lib()).dsa_rope_qkv656(
        ctypes.byref(rope), _arg_strided(positions, "positions", torch.int32, (rope.n_axes, T), dev), st(positions, 0), T, H,
        _arg_strided(q_nope, "q_nope", bf, (T, H, 512), dev), st(q_nope, 0), st(q_nope, 1),
        _arg_strided(q_pe, "q_pe", bf, (T, H, 64), dev), st(q_pe, 0), st(q_pe, 1),
        None if q_out is None else _arg(q_out, "q_out", bf, (T, H, 576), dev),
        _arg_strided(kv_c, "kv_c", bf, (T, 512), dev), st(kv_c, 0), _arg_strided(k_pe, "k_pe", bf, (T, 64), dev), st(k_pe, 0),
        None if slots is None else _arg(slots, "slots", torch.int64, (T,), dev),
        None if pool is None else _arg(pool, "pool", torch.uint8, (_dims(pool, "pool", 2)[0], 656), dev),
        0 if pool is None else pool.shape[0], _flag(err_flag, dev), s), "dsa_rope_qkv656")


def dsa_chunk_attn_workspace_bytes(T: int, H: int, B: int, layout) -> int:
    return int(lib().dsa_chunk_attn_workspace_bytes(T, H, B, LAYOUTS.get(layout, layout)))


def chunk_workspace_for(T: int, H: int, B: int, layout, device=None) -> torch.Tensor:
    """A device workspace for dsa_chunk_attn of up to T tokens of up to B requests, with up to H heads."""
    return torch.empty(dsa_chunk_attn_workspace_bytes(T, H, B, layout), dtype=torch.uint8, device=device or "cuda")


def dsa_chunk_attn(q_bf16, pool, layout, page_table, page_size, cu_q, kv_lens, sm_scale, o, lse, workspace,
                   causal=True, err_flag=None, stream=None) -> None:
    """Dense attention of each request's new tokens, q [T, H, 512 or 576] rows cu_q[b]:cu_q[b + 1], over its
    kv_lens[b] rows of the paged pool (see include/dsa.h)."""
    dev, s = _call_device(stream)
    lay = LAYOUTS.get(layout, layout)
    T, H, D = _dims(q_bf16, "q_bf16", 3)
    B, W = _dims(page_table, "page_table", 2)
    rows, _ = _dims(pool, "pool", 2)
    i32 = torch.int32
    _check((_lib or lib()).dsa_chunk_attn(
        _arg(q_bf16, "q_bf16", torch.bfloat16, None, dev), T, H, D, _arg(pool, "pool", torch.uint8, None, dev), rows, lay,
        _kv_row_dim(pool, lay), _arg(page_table, "page_table", i32, None, dev), B, W, page_size,
        _arg(cu_q, "cu_q", i32, (B + 1,), dev), _arg(kv_lens, "kv_lens", i32, (B,), dev), int(causal), sm_scale,
        _arg(o, "o", torch.bfloat16, (T, H, 512), dev), _arg(lse, "lse", torch.float32, (T, H), dev),
        _arg(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _flag(err_flag, dev), s), "dsa_chunk_attn")


def dsa_prefix_attn_workspace_bytes(T: int, H: int, B: int, layout) -> int:
    return int(lib().dsa_prefix_attn_workspace_bytes(T, H, B, LAYOUTS.get(layout, layout)))


def prefix_workspace_for(T: int, H: int, B: int, layout, device=None) -> torch.Tensor:
    """A device workspace for dsa_prefix_attn of up to T tokens of up to B requests, with up to H heads."""
    return torch.empty(dsa_prefix_attn_workspace_bytes(T, H, B, layout), dtype=torch.uint8, device=device or "cuda")


def dsa_prefix_attn(q_bf16, pool, layout, page_table, page_size, cu_q, kv_lens, group_cu, prefix_lens, sm_scale, o, lse,
                    workspace, causal=True, err_flag=None, stream=None) -> None:
    """dsa_chunk_attn for requests that begin with common rows: group g's requests group_cu[g]:group_cu[g + 1] share their
    first prefix_lens[g] keys, which are read once for all of them (see include/dsa.h)."""
    dev, s = _call_device(stream)
    lay = LAYOUTS.get(layout, layout)
    T, H, D = _dims(q_bf16, "q_bf16", 3)
    B, W = _dims(page_table, "page_table", 2)
    rows, _ = _dims(pool, "pool", 2)
    G, = _dims(prefix_lens, "prefix_lens", 1)
    i32 = torch.int32
    _check((_lib or lib()).dsa_prefix_attn(
        _arg(q_bf16, "q_bf16", torch.bfloat16, None, dev), T, H, D, _arg(pool, "pool", torch.uint8, None, dev), rows, lay,
        _kv_row_dim(pool, lay), _arg(page_table, "page_table", i32, None, dev), B, W, page_size,
        _arg(cu_q, "cu_q", i32, (B + 1,), dev), _arg(kv_lens, "kv_lens", i32, (B,), dev),
        _arg(group_cu, "group_cu", i32, (G + 1,), dev), _arg(prefix_lens, "prefix_lens", i32, (G,), dev), G, int(causal), sm_scale,
        _arg(o, "o", torch.bfloat16, (T, H, 512), dev), _arg(lse, "lse", torch.float32, (T, H), dev),
        _arg(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), _flag(err_flag, dev), s), "dsa_prefix_attn")
