"""ctypes binding of libqg (include/qg.h): the same entry points, the same
argument order. It only marshals arguments; every step of the computation
runs in the library's HIP kernels.

Buffers may be passed as torch tensors (their device pointer is used) or as
integer device addresses. ``stream=None`` means torch's current stream.
Non-zero status codes raise ``QGError``.
"""
from __future__ import annotations

import ctypes
import os

QG_I8_ROW, QG_U4_G64, QG_B1_G128, QG_I8_G64 = 1, 2, 3, 4
QG_OP_GEMV, QG_OP_GEMM, QG_OP_GEMV_ARGMAX = 1, 2, 3
QG_OK = 0
QG_ERR_NULL, QG_ERR_FORMAT, QG_ERR_SHAPE, QG_ERR_ALIGN = -1, -2, -3, -4
QG_ERR_WORKSPACE, QG_ERR_ALIAS, QG_ERR_LAUNCH, QG_ERR_UNSUPPORTED = -5, -6, -7, -8
QG_ERR_SCRATCH = -9
QG_STATIC_SCRATCH_BYTES = 8 << 20
QG_MAX_GEMV_BATCH = 16
QG_MAX_ARGMAX_BATCH = 256
QG_WS_CONTROL_BYTES = 8192
QG_F32, QG_BF16 = 1, 2
QG_MAX_PLAN_BATCH = 8192
QG_MAX_TOP = 64

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqg.so")

EXPORTS = ("qgemv", "qgemm", "qgemv_argmax", "qgemv_argmax_noalloc", "qembed",
           "qg_workspace_bytes", "qg_status_str", "qg_abi_version",
           "qkv_cache_bytes", "qkv_plan", "qkv_append", "qkv_read", "qkv_attn",
           "qkv_attn_workspace_bytes", "qlogprobs", "qlogprobs_workspace_bytes")

_lib = None


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class KVCache:
    """The paged 4-bit key/value cache as the entry points take it
    (qg_kv_cache): its device memory (a tensor, kept alive here, or an
    address) and its geometry. `tensors.kv_cache` allocates one."""

    def __init__(self, data, num_pages, page_size, kv_heads, head_dim):
        self.data = data
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.kv_heads, self.head_dim = int(kv_heads), int(head_dim)
        self._struct = _KVCacheStruct(_ptr(data), self.num_pages, self.page_size, self.kv_heads, self.head_dim)
        self._ref = ctypes.byref(self._struct)
        need = lib().qkv_cache_bytes(self._ref)
        if data is not None and not isinstance(data, int) and not data.is_contiguous():
            raise ValueError("the cache's memory is not contiguous")
        if need and data is not None and not isinstance(data, int) and data.numel() * data.element_size() < need:
            raise ValueError(f"the cache's memory has {data.numel() * data.element_size()} bytes, its geometry needs {need}")


class QGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if it has not been built: there is no
    other implementation to fall back to."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gemm_qgemv_amd.build` (or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        L.qgemv.argtypes = [I32, P, P, P, P, P, I64, I64, I32, P, SZ, P]
        L.qgemm.argtypes = [I32, P, P, P, P, P, I64, I64, I64, P, SZ, P]
        L.qgemv_argmax.argtypes = [I32, P, P, P, P, P, P, I64, I64, I32, P, SZ, P]
        L.qgemv_argmax_noalloc.argtypes = [I32, P, P, P, P, P, P, I64, I64, I32, P]
        L.qembed.argtypes = [I32, P, P, P, P, P, I64, I64, I64, P]
        L.qg_workspace_bytes.argtypes = [I32, I32, I64, I64, I64]
        L.qg_workspace_bytes.restype = SZ
        L.qg_status_str.argtypes = [I32]
        L.qg_status_str.restype = ctypes.c_char_p
        L.qg_abi_version.argtypes = []
        F = ctypes.c_float
        L.qkv_cache_bytes.argtypes = [P]
        L.qkv_plan.argtypes = [P, P, P, I32, I32, P, I64, P, I64, P, P, P, P, P, P, I64, P, P]
        L.qkv_append.argtypes = [I32, P, I64, P, I64, P, I64, P, P]
        L.qkv_read.argtypes = [I32, P, P, I64, P, I64, P, I64, P]
        L.qkv_attn.argtypes = [I32, P, I64, P, P, I64, P, P, I32, I64, I64, I64, I32, F, I64, P, I64, P,
                               P, SZ, P]
        L.qkv_attn_workspace_bytes.argtypes = [P, I32, I64, I64, I64, I32]
        L.qlogprobs.argtypes = [P, I64, I64, I64, P, I32, P, P, P, P, P, P, SZ, P]
        L.qlogprobs_workspace_bytes.argtypes = [I64, I64, I32]
        for f in (L.qkv_cache_bytes, L.qkv_attn_workspace_bytes, L.qlogprobs_workspace_bytes):
            f.restype = SZ
        for f in (L.qgemv, L.qgemm, L.qgemv_argmax, L.qgemv_argmax_noalloc, L.qembed,
                  L.qg_abi_version, L.qkv_plan, L.qkv_append, L.qkv_read, L.qkv_attn, L.qlogprobs):
            f.restype = I32
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    try:                         # the common case first: a call passes up to 12 tensors
        return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):   # an address
            return t
        raise TypeError(f"a tensor or a device address is needed, not {type(t).__name__}") from None


_current_stream = None


def _stream(stream):
    if stream is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _raw_stream_lookup()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _raw_stream_lookup():
    """A function that gives the address of torch's current stream. Through
    torch.cuda.current_stream() that takes some 2 us of host time a call,
    as much as a small kernel; the raw lookup takes 0.2."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(torch.cuda.current_device())


def _nbytes(ws, ws_bytes):
    if ws_bytes is not None:
        return int(ws_bytes)
    if ws is None or isinstance(ws, int):
        return 0
    return ws.numel() * ws.element_size()


def _check(status, where):
    if status != QG_OK:
        raise QGError(status, where)


def qgemv(fmt, codes, scales, biases, x, y, M, K, batch, ws=None, ws_bytes=None, stream=None):
    _check(lib().qgemv(fmt, _ptr(codes), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y),
                       M, K, batch, _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)), "qgemv")


def qgemm(fmt, codes, scales, biases, x, y, M, K, N, ws=None, ws_bytes=None, stream=None):
    _check(lib().qgemm(fmt, _ptr(codes), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y),
                       M, K, N, _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)), "qgemm")


def qgemv_argmax(fmt, codes, scales, biases, x, logits, idx, M, K, batch, ws=None,
                 ws_bytes=None, stream=None):
    _check(lib().qgemv_argmax(fmt, _ptr(codes), _ptr(scales), _ptr(biases), _ptr(x),
                              _ptr(logits), _ptr(idx), M, K, batch, _ptr(ws),
                              _nbytes(ws, ws_bytes), _stream(stream)), "qgemv_argmax")


def qgemv_argmax_noalloc(fmt, codes, scales, biases, x, logits, idx, M, K, batch, stream=None):
    _check(lib().qgemv_argmax_noalloc(fmt, _ptr(codes), _ptr(scales), _ptr(biases), _ptr(x),
                                      _ptr(logits), _ptr(idx), M, K, batch, _stream(stream)),
           "qgemv_argmax_noalloc")


def qembed(fmt, codes, scales, biases, ids, out, M, K, n, stream=None):
    _check(lib().qembed(fmt, _ptr(codes), _ptr(scales), _ptr(biases), _ptr(ids), _ptr(out),
                        M, K, n, _stream(stream)), "qembed")


def qkv_cache_bytes(cache) -> int:
    return int(lib().qkv_cache_bytes(cache._ref))


def qkv_plan(len_old, keep, n_new, batch, page_size, block_table, table_stride, ring, ring_size, state_in,
             state_out, kv_len, cu_q, slots, pos, total, denied, stream=None):
    _check(lib().qkv_plan(_ptr(len_old), _ptr(keep), _ptr(n_new), batch, page_size, _ptr(block_table), table_stride,
                          _ptr(ring), ring_size, _ptr(state_in), _ptr(state_out), _ptr(kv_len), _ptr(cu_q),
                          _ptr(slots), _ptr(pos), total, _ptr(denied), _stream(stream)), "qkv_plan")


def qkv_append(dtype, k, k_stride, v, v_stride, slots, n, cache, stream=None):
    _check(lib().qkv_append(dtype, _ptr(k), k_stride, _ptr(v), v_stride, _ptr(slots), n, cache._ref,
                            _stream(stream)), "qkv_append")


def qkv_read(dtype, cache, slots, n, k, k_stride, v, v_stride, stream=None):
    _check(lib().qkv_read(dtype, cache._ref, _ptr(slots), n, _ptr(k), k_stride, _ptr(v), v_stride,
                          _stream(stream)), "qkv_read")


def qkv_attn(dtype, q, q_stride, cache, block_table, table_stride, cu_q, kv_len, batch, total_q, max_q, max_kv,
             q_heads, scale, window, out, out_stride, lse=None, ws=None, ws_bytes=None, stream=None):
    _check(lib().qkv_attn(dtype, _ptr(q), q_stride, cache._ref, _ptr(block_table), table_stride, _ptr(cu_q),
                          _ptr(kv_len), batch, total_q, max_q, max_kv, q_heads, scale, window, _ptr(out),
                          out_stride, _ptr(lse), _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)), "qkv_attn")


def qkv_attn_workspace_bytes(cache, batch, total_q, max_q, max_kv, q_heads) -> int:
    return int(lib().qkv_attn_workspace_bytes(cache._ref, batch, total_q, max_q, max_kv, q_heads))


def qlogprobs(logits, ld, rows, vocab, ids, top, logprob, entropy, rank, top_ids=None, top_logprobs=None,
              ws=None, ws_bytes=None, stream=None):
    _check(lib().qlogprobs(_ptr(logits), ld, rows, vocab, _ptr(ids), top, _ptr(logprob), _ptr(entropy), _ptr(rank),
                           _ptr(top_ids), _ptr(top_logprobs), _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)),
           "qlogprobs")


def qlogprobs_workspace_bytes(rows, vocab, top) -> int:
    return int(lib().qlogprobs_workspace_bytes(rows, vocab, top))


def qg_workspace_bytes(op, fmt, M, K, rows) -> int:
    return int(lib().qg_workspace_bytes(op, fmt, M, K, rows))


def qg_status_str(status) -> str:
    return lib().qg_status_str(status).decode()


def status_str(status) -> str:
    try:
        return qg_status_str(status)
    except Exception:  # library missing: still name the code
        return f"status {status}"


def qg_abi_version() -> int:
    return int(lib().qg_abi_version())
