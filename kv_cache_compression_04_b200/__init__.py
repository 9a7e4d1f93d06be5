"""Python binding of libkvc.so, the B200 (sm_100a) KV-cache codec.

Argument marshalling only: every step of the codec runs in the library's CUDA
kernels; PyTorch supplies device memory and streams. The names mirror the C
ABI in ``include/kvc.h`` (``kvc_compress``, ``kvc_decompress``,
``kvc_max_compressed_bytes``, ``kvc_workspace_bytes``, ``kvc_stream_status``,
``kvc_status_string``). If ``libkvc.so`` has not been built, importing the
library raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkvc.so")

KVC_DENSE, KVC_PAGED = 0, 1
KVC_MAX_REQUESTS = 1024
KVC_NOALLOC_SCRATCH_BYTES = 16 << 20
STATUS = ["KVC_OK", "KVC_ERR_INVALID_ARG", "KVC_ERR_UNSUPPORTED", "KVC_ERR_CAPACITY",
          "KVC_ERR_NONFINITE", "KVC_ERR_RANGE", "KVC_ERR_CORRUPT", "KVC_ERR_TIMEOUT",
          "KVC_ERR_CUDA"]
(KVC_OK, KVC_ERR_INVALID_ARG, KVC_ERR_UNSUPPORTED, KVC_ERR_CAPACITY, KVC_ERR_NONFINITE,
 KVC_ERR_RANGE, KVC_ERR_CORRUPT, KVC_ERR_TIMEOUT, KVC_ERR_CUDA) = range(9)

# Every symbol include/kvc.h declares.
EXPORTS = ["kvc_max_compressed_bytes", "kvc_workspace_bytes", "kvc_compress",
           "kvc_decompress", "kvc_stream_status", "kvc_status_string", "kvc_compress_noalloc",
           "kvc_decompress_workspace_bytes", "kvc_unfused_workspace_bytes",
           "kvc_compress_unfused", "kvc_test_compress_stalled", "kvc_compress_timed",
           "kvc_decompress_timed", "kvc_attend_workspace_bytes", "kvc_attend",
           "kvc_attend_timed", "kvc_cache_block_bytes", "kvc_cache_stream_seed",
           "kvc_cache_status_clear", "kvc_cache_write", "kvc_cache_read",
           "kvc_cache_load_workspace_bytes", "kvc_cache_load", "kvc_cache_load_noting",
           "kvc_cache_attend_workspace_bytes", "kvc_cache_attend", "kvc_test_e2m1", "kvc_test_div_const",
           "kvc_test_rcp_scale"]


class KvcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS[status] if 0 <= status < len(STATUS) else status}")


class kvc_params(C.Structure):
    _fields_ = [("bits", C.c_int32), ("group_size", C.c_int32), ("sign_seed", C.c_uint64),
                ("lossless", C.c_int32), ("quant", C.c_int32), ("signs", C.c_int32),
                ("reserved", C.c_int32)]


# Quantizers (kvc_params.quant) and sign diagonals (kvc_params.signs).
KVC_QUANT_ASYM, KVC_QUANT_SYM, KVC_QUANT_FP4 = 0, 1, 2
KVC_SIGNS_GLOBAL, KVC_SIGNS_PER_VECTOR = 0, 1


# Lossless-stage modes (kvc_params.lossless) and pipeline ids of a chunk.
KVC_LOSSLESS_FIXED, KVC_LOSSLESS_SEARCH, KVC_LOSSLESS_NONE = range(3)


class kvc_attn_desc(C.Structure):
    _fields_ = [("layers", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("q_per_kv", C.c_int32), ("bits", C.c_int32), ("group_size", C.c_int32),
                ("quant", C.c_int32), ("kernel", C.c_int32), ("n_requests", C.c_int32),
                ("scale", C.c_float),
                ("seq_lens", C.POINTER(C.c_int32)), ("q", C.c_void_p), ("out", C.c_void_p)]


# Element types of the paged cache's rows, queries and outputs.
KVC_BF16, KVC_FP16 = 0, 1
KVC_CACHE_MAX_Q_PER_KV = 64


class kvc_cache_desc(C.Structure):
    _fields_ = [("layers", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("bits", C.c_int32), ("group_size", C.c_int32), ("quant", C.c_int32),
                ("signs", C.c_int32), ("first_layer", C.c_int32), ("sign_seed", C.c_uint64),
                ("page_tokens", C.c_int32), ("reserved", C.c_int32), ("num_pages", C.c_int64),
                ("pool", C.c_void_p), ("stride_layer", C.c_int64), ("stride_page", C.c_int64),
                ("stride_kv", C.c_int64), ("stride_head", C.c_int64)]


class kvc_cache_rows(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("reserved", C.c_int32), ("tokens", C.c_int64),
                ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_stride_layer", C.c_int64), ("k_stride_token", C.c_int64),
                ("k_stride_head", C.c_int64), ("v_stride_layer", C.c_int64),
                ("v_stride_token", C.c_int64), ("v_stride_head", C.c_int64),
                ("slots", C.c_void_p)]


class kvc_cache_attn(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("q_per_kv", C.c_int32), ("n_requests", C.c_int32),
                ("max_q", C.c_int32), ("causal", C.c_int32), ("window", C.c_int32),
                ("scale", C.c_float), ("reserved", C.c_int32), ("q_tokens", C.c_int64),
                ("q_starts", C.c_void_p), ("seq_lens", C.c_void_p), ("page_table", C.c_void_p),
                ("page_table_pages", C.c_int64), ("page_table_stride", C.c_int64),
                ("q", C.c_void_p),
                ("q_stride_layer", C.c_int64), ("q_stride_token", C.c_int64),
                ("q_stride_head", C.c_int64), ("out", C.c_void_p),
                ("out_stride_layer", C.c_int64), ("out_stride_token", C.c_int64),
                ("out_stride_head", C.c_int64), ("lse", C.c_void_p)]


class kvc_kv_desc(C.Structure):
    _fields_ = [("kind", C.c_int32), ("layers", C.c_int32), ("kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("data", C.c_void_p),
                ("stride_layer", C.c_int64), ("stride_kv", C.c_int64),
                ("stride_head", C.c_int64), ("tokens", C.c_int64),
                ("stride_token", C.c_int64), ("page_tokens", C.c_int32),
                ("n_requests", C.c_int32), ("stride_page", C.c_int64),
                ("stride_slot", C.c_int64), ("num_pages", C.c_int64),
                ("seq_lens", C.POINTER(C.c_int32)), ("page_table", C.c_void_p),
                ("page_table_stride", C.c_int64)]


_lib = None


def lib() -> C.CDLL:
    """The loaded libkvc.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libkvc.so is not built ({LIB_PATH}); run "
                              "`python -m kv_cache_compression_04_b200.build`")
        L = C.CDLL(LIB_PATH)
        D, P = C.POINTER(kvc_kv_desc), C.POINTER(kvc_params)
        L.kvc_max_compressed_bytes.restype = C.c_size_t
        L.kvc_max_compressed_bytes.argtypes = [D, P]
        L.kvc_workspace_bytes.restype = C.c_size_t
        L.kvc_workspace_bytes.argtypes = [D, P]
        L.kvc_decompress_workspace_bytes.restype = C.c_size_t
        L.kvc_decompress_workspace_bytes.argtypes = [D]
        L.kvc_compress.restype = C.c_int
        L.kvc_compress.argtypes = [D, P, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p,
                                   C.c_size_t, C.c_void_p]
        L.kvc_decompress.restype = C.c_int
        L.kvc_decompress.argtypes = [C.c_void_p, C.c_size_t, D, C.c_void_p, C.c_size_t,
                                     C.c_void_p]
        L.kvc_stream_status.restype = C.c_int
        L.kvc_stream_status.argtypes = [C.c_void_p, C.c_void_p]
        L.kvc_status_string.restype = C.c_char_p
        L.kvc_status_string.argtypes = [C.c_int]
        L.kvc_compress_noalloc.restype = C.c_int
        L.kvc_compress_noalloc.argtypes = [D, P, C.c_void_p, C.c_size_t, C.c_void_p,
                                           C.c_void_p, C.c_void_p]
        L.kvc_unfused_workspace_bytes.restype = C.c_size_t
        L.kvc_unfused_workspace_bytes.argtypes = [D, P]
        L.kvc_compress_unfused.restype = C.c_int
        L.kvc_compress_unfused.argtypes = [D, P, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p,
                                           C.c_size_t, C.c_void_p]
        L.kvc_compress_timed.restype = C.c_int
        L.kvc_compress_timed.argtypes = [D, P, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p,
                                         C.c_size_t, C.POINTER(C.c_void_p), C.c_int, C.c_void_p]
        L.kvc_decompress_timed.restype = C.c_int
        L.kvc_decompress_timed.argtypes = [C.c_void_p, C.c_size_t, D, C.c_void_p, C.c_size_t,
                                           C.POINTER(C.c_void_p), C.c_int, C.c_void_p]
        A = C.POINTER(kvc_attn_desc)
        L.kvc_attend_workspace_bytes.restype = C.c_size_t
        L.kvc_attend_workspace_bytes.argtypes = [A]
        L.kvc_attend.restype = C.c_int
        L.kvc_attend.argtypes = [C.c_void_p, C.c_size_t, A, C.c_void_p, C.c_size_t, C.c_void_p]
        L.kvc_attend_timed.restype = C.c_int
        L.kvc_attend_timed.argtypes = [C.c_void_p, C.c_size_t, A, C.c_void_p, C.c_size_t,
                                       C.POINTER(C.c_void_p), C.c_int, C.c_void_p]
        K, R, T = C.POINTER(kvc_cache_desc), C.POINTER(kvc_cache_rows), C.POINTER(kvc_cache_attn)
        for name, res, args in (
                ("kvc_cache_block_bytes", C.c_size_t, [K]),
                ("kvc_cache_stream_seed", C.c_uint64, [K]),
                ("kvc_cache_status_clear", C.c_int, [C.c_void_p, C.c_void_p]),
                ("kvc_cache_write", C.c_int, [K, R, C.c_void_p, C.c_void_p]),
                ("kvc_cache_read", C.c_int, [K, R, C.c_void_p, C.c_void_p]),
                ("kvc_cache_load_workspace_bytes", C.c_size_t, [K, C.POINTER(C.c_int32), C.c_int32]),
                ("kvc_cache_load", C.c_int, [C.c_void_p, C.c_size_t, K, C.POINTER(C.c_int32),
                                             C.c_int32, C.c_void_p, C.c_void_p, C.c_size_t,
                                             C.c_void_p]),
                ("kvc_cache_load_noting", C.c_int, [C.c_void_p, C.c_size_t, K, C.POINTER(C.c_int32),
                                                    C.c_int32, C.c_void_p, C.c_void_p, C.c_size_t,
                                                    C.c_void_p, C.c_void_p]),
                ("kvc_cache_attend_workspace_bytes", C.c_size_t, [K, T]),
                ("kvc_cache_attend", C.c_int, [K, T, C.c_void_p, C.c_size_t, C.c_void_p,
                                               C.c_void_p])):
            getattr(L, name).restype = res
            getattr(L, name).argtypes = args
        L.kvc_test_e2m1.restype = C.c_int
        L.kvc_test_e2m1.argtypes = [C.c_void_p, C.c_void_p, C.c_uint64, C.c_void_p]
        L.kvc_test_div_const.restype = C.c_int
        L.kvc_test_div_const.argtypes = [C.c_void_p, C.c_void_p, C.c_uint64, C.c_int, C.c_void_p]
        L.kvc_test_rcp_scale.restype = C.c_int
        L.kvc_test_rcp_scale.argtypes = [C.c_void_p, C.c_void_p, C.c_uint64, C.c_void_p]
        L.kvc_test_compress_stalled.restype = C.c_int
        L.kvc_test_compress_stalled.argtypes = [D, P, C.c_void_p, C.c_size_t, C.c_void_p,
                                                C.c_void_p, C.c_size_t, C.c_uint32, C.c_uint64,
                                                C.c_void_p]
        _lib = L
    return _lib


# ---------------------------------------------------------------- raw ABI --
def kvc_max_compressed_bytes(desc: kvc_kv_desc, params: kvc_params) -> int:
    return lib().kvc_max_compressed_bytes(C.byref(desc), C.byref(params))


def kvc_workspace_bytes(desc: kvc_kv_desc, params: kvc_params) -> int:
    return lib().kvc_workspace_bytes(C.byref(desc), C.byref(params))


def kvc_decompress_workspace_bytes(desc: kvc_kv_desc) -> int:
    return lib().kvc_decompress_workspace_bytes(C.byref(desc))


def kvc_compress(desc, params, out_ptr, out_capacity, out_bytes_dev_ptr, ws_ptr, ws_bytes,
                 stream) -> int:
    return lib().kvc_compress(C.byref(desc), C.byref(params), out_ptr, out_capacity,
                              out_bytes_dev_ptr, ws_ptr, ws_bytes, stream)


def kvc_unfused_workspace_bytes(desc: kvc_kv_desc, params: kvc_params) -> int:
    return lib().kvc_unfused_workspace_bytes(C.byref(desc), C.byref(params))


def kvc_compress_unfused(desc, params, out_ptr, out_capacity, out_bytes_dev_ptr, ws_ptr, ws_bytes,
                         stream) -> int:
    return lib().kvc_compress_unfused(C.byref(desc), C.byref(params), out_ptr, out_capacity,
                                      out_bytes_dev_ptr, ws_ptr, ws_bytes, stream)


def kvc_compress_noalloc(desc, params, out_ptr, out_capacity, out_bytes_dev_ptr, status_dev_ptr,
                         stream) -> int:
    return lib().kvc_compress_noalloc(C.byref(desc), C.byref(params), out_ptr, out_capacity,
                                      out_bytes_dev_ptr, status_dev_ptr, stream)


def kvc_test_compress_stalled(desc, params, out_ptr, out_capacity, out_bytes_dev_ptr, ws_ptr,
                              ws_bytes, skip_chunks, wait_ns, stream) -> int:
    """Test-only (include/kvc_test.h): kvc_compress whose compaction skips
    `skip_chunks` chunks and gives up its waits after `wait_ns`."""
    return lib().kvc_test_compress_stalled(C.byref(desc), C.byref(params), out_ptr, out_capacity,
                                           out_bytes_dev_ptr, ws_ptr, ws_bytes, skip_chunks,
                                           wait_ns, stream)


def _event_array(events):
    """torch.cuda.Event objects -> a C array of their cudaEvent_t handles."""
    return (C.c_void_p * len(events))(*[e.cuda_event for e in events])


def kvc_compress_timed(desc, params, out_ptr, out_capacity, out_bytes_dev_ptr, ws_ptr, ws_bytes,
                       events, stream) -> int:
    """kvc_compress recording `events` (5 torch.cuda.Event, created with
    enable_timing=True and already created on the device) around its kernels."""
    arr = _event_array(events)
    return lib().kvc_compress_timed(C.byref(desc), C.byref(params), out_ptr, out_capacity,
                                    out_bytes_dev_ptr, ws_ptr, ws_bytes, arr, len(events), stream)


def kvc_decompress_timed(in_ptr, in_bytes, desc, ws_ptr, ws_bytes, events, stream) -> int:
    arr = _event_array(events)
    return lib().kvc_decompress_timed(in_ptr, in_bytes, C.byref(desc), ws_ptr, ws_bytes, arr,
                                      len(events), stream)


def attn_desc(layers, kv_heads, q_per_kv, bits, group, seq_lens, q, out, scale,
              head_dim: int = 128, quant: int = 0, kernel: int = 0) -> kvc_attn_desc:
    """Descriptor of kvc_attend: q bf16 [layers, n_requests, kv_heads * q_per_kv,
    head_dim] and out fp32 of the same shape (device tensors)."""
    seq = (C.c_int32 * max(len(seq_lens), 1))(*[int(x) for x in seq_lens])
    d = kvc_attn_desc(layers, kv_heads, head_dim, q_per_kv, bits, group, quant, kernel,
                      len(seq_lens), float(scale), C.cast(seq, C.POINTER(C.c_int32)), q.data_ptr(),
                      out.data_ptr())
    d._keep = (seq, q, out)
    return d


def kvc_attend_workspace_bytes(attn: kvc_attn_desc) -> int:
    return lib().kvc_attend_workspace_bytes(C.byref(attn))


def kvc_attend(in_ptr, in_bytes, attn, ws_ptr, ws_bytes, stream) -> int:
    return lib().kvc_attend(in_ptr, in_bytes, C.byref(attn), ws_ptr, ws_bytes, stream)


def kvc_attend_timed(in_ptr, in_bytes, attn, ws_ptr, ws_bytes, events, stream) -> int:
    arr = _event_array(events)
    return lib().kvc_attend_timed(in_ptr, in_bytes, C.byref(attn), ws_ptr, ws_bytes, arr,
                                  len(events), stream)


def kvc_decompress(in_ptr, in_bytes, desc, ws_ptr, ws_bytes, stream) -> int:
    return lib().kvc_decompress(in_ptr, in_bytes, C.byref(desc), ws_ptr, ws_bytes, stream)


def kvc_stream_status(ws_ptr, stream) -> int:
    return lib().kvc_stream_status(ws_ptr, stream)


def kvc_status_string(status: int) -> str:
    return lib().kvc_status_string(status).decode()


def kvc_cache_block_bytes(cache: kvc_cache_desc) -> int:
    return lib().kvc_cache_block_bytes(C.byref(cache))


def kvc_cache_stream_seed(cache: kvc_cache_desc) -> int:
    return lib().kvc_cache_stream_seed(C.byref(cache))


def kvc_cache_status_clear(status_ptr, stream) -> int:
    return lib().kvc_cache_status_clear(status_ptr, stream)


def kvc_cache_write(cache, rows, status_ptr, stream) -> int:
    return lib().kvc_cache_write(C.byref(cache), C.byref(rows), status_ptr, stream)


def kvc_cache_read(cache, rows, status_ptr, stream) -> int:
    return lib().kvc_cache_read(C.byref(cache), C.byref(rows), status_ptr, stream)


def kvc_cache_load_workspace_bytes(cache, seq_lens) -> int:
    arr = (C.c_int32 * max(len(seq_lens), 1))(*seq_lens)
    return lib().kvc_cache_load_workspace_bytes(C.byref(cache), arr, len(seq_lens))


def kvc_cache_load(in_ptr, in_bytes, cache, seq_lens, slots_ptr, ws_ptr, ws_bytes, stream) -> int:
    arr = (C.c_int32 * max(len(seq_lens), 1))(*seq_lens)
    return lib().kvc_cache_load(in_ptr, in_bytes, C.byref(cache), arr, len(seq_lens), slots_ptr,
                                ws_ptr, ws_bytes, stream)


def kvc_cache_load_noting(in_ptr, in_bytes, cache, seq_lens, slots_ptr, ws_ptr, ws_bytes, status_ptr,
                          stream) -> int:
    arr = (C.c_int32 * max(len(seq_lens), 1))(*seq_lens)
    return lib().kvc_cache_load_noting(in_ptr, in_bytes, C.byref(cache), arr, len(seq_lens), slots_ptr,
                                       ws_ptr, ws_bytes, status_ptr, stream)


def kvc_cache_attend_workspace_bytes(cache, attn) -> int:
    return lib().kvc_cache_attend_workspace_bytes(C.byref(cache), C.byref(attn))


def kvc_cache_attend(cache, attn, ws_ptr, ws_bytes, status_ptr, stream) -> int:
    return lib().kvc_cache_attend(C.byref(cache), C.byref(attn), ws_ptr, ws_bytes, status_ptr,
                                  stream)


# ------------------------------------------------------- descriptor helpers --
def params(bits: int, group: int, sign_seed: int = 0, lossless: int = KVC_LOSSLESS_FIXED,
           quant: int = KVC_QUANT_ASYM, signs: int = KVC_SIGNS_GLOBAL) -> kvc_params:
    return kvc_params(bits, group, sign_seed, lossless, quant, signs, 0)


def dense_desc(kv) -> kvc_kv_desc:
    """Descriptor of a bf16 tensor shaped [layers, 2, kv_heads, tokens, head_dim]
    (any strides with head_dim contiguous)."""
    L, two, H, T, D = kv.shape
    assert two == 2 and kv.stride(4) == 1, "expects [layers, 2, kv_heads, tokens, head_dim]"
    d = kvc_kv_desc()
    d.kind, d.layers, d.kv_heads, d.head_dim = KVC_DENSE, L, H, D
    d.data = kv.data_ptr() if kv.numel() else None
    d.stride_layer, d.stride_kv, d.stride_head = kv.stride(0), kv.stride(1), kv.stride(2)
    d.tokens, d.stride_token = T, kv.stride(3)
    d._keep = (kv,)
    return d


def paged_desc(pool, page_table, seq_lens, kv_heads: int | None = None) -> kvc_kv_desc:
    """Descriptor of a page pool shaped [layers, pages, 2, kv_heads, page_tokens,
    head_dim] with an int32 device page table [n_requests, max_pages] and a host
    list of per-request token counts."""
    L, P, two, H, PT, D = pool.shape
    assert two == 2 and pool.stride(5) == 1
    seq = (C.c_int32 * max(len(seq_lens), 1))(*[int(x) for x in seq_lens])
    d = kvc_kv_desc()
    d.kind, d.layers, d.kv_heads, d.head_dim = KVC_PAGED, L, H if kv_heads is None else kv_heads, D
    d.data = pool.data_ptr()
    d.stride_layer, d.stride_page, d.stride_kv = pool.stride(0), pool.stride(1), pool.stride(2)
    d.stride_head, d.stride_slot = pool.stride(3), pool.stride(4)
    d.page_tokens, d.n_requests, d.num_pages = PT, len(seq_lens), P
    d.seq_lens = C.cast(seq, C.POINTER(C.c_int32))
    d.page_table = page_table.data_ptr()
    d.page_table_stride = page_table.stride(0)
    d._keep = (pool, page_table, seq)
    return d


def _stream_ptr(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != KVC_OK:
        raise KvcError(status, where)


# --------------------------------------------------------- convenience API --
class Codec:
    """Compresses / decompresses KV caches with caller-visible buffers.

    Buffers come from PyTorch's caching allocator (plumbing only); every
    compute step runs in libkvc's kernels. Errors raise KvcError."""

    def __init__(self, bits: int = 4, group: int = 128, sign_seed: int = 0,
                 lossless: int = KVC_LOSSLESS_FIXED, quant: int = KVC_QUANT_ASYM,
                 signs: int = KVC_SIGNS_GLOBAL):
        self.params = params(bits, group, sign_seed, lossless, quant, signs)

    def buffers(self, desc: kvc_kv_desc, device="cuda"):
        import torch
        cap = kvc_max_compressed_bytes(desc, self.params)
        wsb = kvc_workspace_bytes(desc, self.params)
        if cap == 0 or wsb == 0:
            raise KvcError(KVC_ERR_INVALID_ARG, "kvc_max_compressed_bytes")
        out = torch.empty(cap, dtype=torch.uint8, device=device)
        # one workspace serves both directions for this shape
        ws = torch.empty(max(wsb, kvc_decompress_workspace_bytes(desc)), dtype=torch.uint8,
                         device=device)
        nbytes = torch.zeros(1, dtype=torch.int64, device=device)
        return out, ws, nbytes

    def compress(self, desc: kvc_kv_desc, out=None, ws=None, nbytes=None, stream=None,
                 check: bool = True):
        """Enqueues compression; returns (out, workspace, device stream length)."""
        if out is None:
            out, ws, nbytes = self.buffers(desc)
        st = kvc_compress(desc, self.params, out.data_ptr(), out.numel(), nbytes.data_ptr(),
                          ws.data_ptr(), ws.numel(), _stream_ptr(stream))
        _check(st, "kvc_compress")
        if check:
            _check(kvc_stream_status(ws.data_ptr(), _stream_ptr(stream)), "kvc_compress (device)")
        return out, ws, nbytes

    @staticmethod
    def decompress(stream_buf, nbytes: int, desc: kvc_kv_desc, ws, stream=None,
                   check: bool = True):
        st = kvc_decompress(stream_buf.data_ptr(), int(nbytes), desc, ws.data_ptr(), ws.numel(),
                            _stream_ptr(stream))
        _check(st, "kvc_decompress")
        if check:
            _check(kvc_stream_status(ws.data_ptr(), _stream_ptr(stream)), "kvc_decompress (device)")


# kvc_cache_rows and kvc_cache_attn as bytes: PagedCache's calls on small batches take as
# long as their host work, and filling a ctypes structure is a third of that.
_ROWS = struct.Struct("<iiqQQ6qQ")
_ATTN = struct.Struct("<6ifiqQQQqqQ3qQ3qQ")


def _raw(name: str, *args):
    """A function of the library under argument types of its own (addresses, bytes)."""
    f = lib()[name]
    f.restype, f.argtypes = C.c_int, args
    return f


def _strides(t):
    """Strides of the first three of four dimensions; of those never stepped along, 0."""
    a, b, c, _ = t.shape
    x, y, z, _ = t.stride()
    return x if a > 1 else 0, y if b > 1 else 0, z if c > 1 else 0


class PagedCache:
    """A KV cache that stays in 4-bit pages on the decode GPU (kvc_cache_* in
    include/kvc.h): ``load`` a received stream, ``write`` new tokens, ``attend``
    over the pages, ``read`` rows back.

    ``pool`` is a uint8 tensor [layers, num_pages, 2, kv_heads, block] (any
    strides but the last, which is 1; made here if not given). ``cache[i]`` and
    ``cache[a:b]`` are views of some layers; rows and queries always have a
    leading layer dimension of that length. Slot numbers are page * page_tokens
    + place in the page.

    Calls are asynchronous on the current stream (or ``stream``). Errors in
    arguments raise at once; data-dependent errors collect in one status word,
    shared by all views, which ``check`` reads (it waits) and clears. Buffers come
    from PyTorch's caching allocator: a workspace grows to the largest call seen
    on its stream and is kept; a captured call has one of the graph's own. Threads
    may share a cache."""

    def __init__(self, layers: int, kv_heads: int, head_dim: int, num_pages: int,
                 page_tokens: int = 16, group: int = 128, sign_seed: int = 0,
                 quant: int = KVC_QUANT_ASYM, signs: int = KVC_SIGNS_GLOBAL, pool=None,
                 device="cuda"):
        import torch
        d = kvc_cache_desc(layers, kv_heads, head_dim, 4, group, quant, signs, 0,
                           sign_seed & (2 ** 64 - 1), page_tokens, 0, num_pages)
        block = kvc_cache_block_bytes(d)
        if block == 0:
            raise KvcError(KVC_ERR_INVALID_ARG, "kvc_cache_block_bytes")
        if pool is None:
            pool = torch.zeros(layers, num_pages, 2, kv_heads, block, dtype=torch.uint8,
                               device=device)
        if (tuple(pool.shape) != (layers, num_pages, 2, kv_heads, block) or not pool.is_cuda or
                pool.dtype != torch.uint8 or (pool.numel() and pool.stride(4) != 1)):
            raise ValueError(f"pool: expects a CUDA uint8 tensor {(layers, num_pages, 2, kv_heads, block)}")
        self.status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self._ws, self._lock = {}, threading.Lock()
        A, N = C.c_void_p, C.c_size_t
        self._calls = (_raw("kvc_cache_write", A, A, A, A), _raw("kvc_cache_read", A, A, A, A),
                       _raw("kvc_cache_attend", A, A, A, N, A, A),
                       {torch.bfloat16: KVC_BF16, torch.float16: KVC_FP16})
        self._set(d, pool)

    def _set(self, d, pool):
        d.layers = pool.shape[0]
        d.pool = pool.data_ptr() if pool.numel() else None
        d.stride_layer, d.stride_page, d.stride_kv, d.stride_head = (
            st if n > 1 else 0 for n, st in zip(pool.shape[:4], pool.stride()))
        self.desc, self.pool, self.device = d, pool, pool.device
        self.index, self._desc, self._status = pool.get_device(), C.addressof(d), self.status.data_ptr()
        self._write, self._read, self._attend, self._types = self._calls
        self._row = (d.layers, d.kv_heads, d.head_dim)

    def __getitem__(self, which) -> "PagedCache":
        if isinstance(which, int):
            if not -self.pool.shape[0] <= which < self.pool.shape[0]:
                raise IndexError(f"layer {which} of {self.pool.shape[0]}")
            which = slice(which, which + 1 or None)
        first, _, step = which.indices(self.pool.shape[0])
        if step != 1:
            raise ValueError("layers are taken in order")
        view = object.__new__(PagedCache)
        view.status, view._ws, view._lock, view._calls = self.status, self._ws, self._lock, self._calls
        d = kvc_cache_desc()
        C.pointer(d)[0] = self.desc
        d.first_layer += first
        view._set(d, self.pool[which])
        return view

    def _here(self, stream, *tensors):
        """The stream's handle, after a look at where the tensors are."""
        import torch
        if torch._C._cuda_getDevice() != self.index:
            raise ValueError(f"the cache is on {self.device}, which is not the current device")
        for t in tensors:
            if t is not None and t.get_device() != self.index:
                raise ValueError(f"a tensor is on {t.device}, the cache on {self.device}")
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.index)
        if stream.device_index != self.index:
            raise ValueError(f"the stream is on device {stream.device_index}, the cache on {self.device}")
        return stream.cuda_stream

    def _may_wait(self, stream, where: str):
        """Waiting for a stream that is being captured would end the capture."""
        import torch
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._may_wait(None, where)
        if torch._C._cuda_isCurrentStreamCapturing():
            raise ValueError(f"{where} waits, which a stream that is being captured cannot")

    def _workspace(self, stream, handle: int, nbytes):
        """The stream's workspace if it has nbytes() (called where that has to be known; 0 for
        arguments that the call then refuses, which no null pointer may hide)."""
        import torch
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._workspace(None, handle, nbytes)
        if torch._C._cuda_isCurrentStreamCapturing():  # a graph's own, from its memory pool
            return torch.empty(max(1, nbytes()), dtype=torch.uint8, device=self.device)
        ws = self._ws.get(handle)
        if ws is None:
            ws = self._ws[handle] = torch.empty(max(1, nbytes()), dtype=torch.uint8, device=self.device)
        return ws

    def _with_workspace(self, where, stream, handle: int, nbytes, call, then=None):
        """call(address, bytes) with a workspace that is large enough (one that is not is
        refused before anything is enqueued, and replaced), then(address) before another
        thread has it."""
        with self._lock:
            ws = self._workspace(stream, handle, nbytes)
            st = call(ws.data_ptr(), ws.numel())
            if st == KVC_ERR_CAPACITY:
                self._ws.pop(handle, None)
                ws = self._workspace(stream, handle, nbytes)
                st = call(ws.data_ptr(), ws.numel())
            if st == KVC_OK and then:
                st = then(ws.data_ptr())
        if st:
            raise KvcError(st, where)

    def _dtype(self, name, t):
        kind = self._types.get(t.dtype)
        if kind is None:
            raise KvcError(KVC_ERR_UNSUPPORTED, f"{name}: {t.dtype}")
        return kind

    def _rows(self, k, v, slots):
        """kvc_cache_rows, as bytes."""
        import torch
        if slots.dtype is not torch.int64 or slots.dim() != 1 or not slots.is_contiguous():
            raise ValueError("slots: expects a contiguous int64 vector")
        n, (layers, heads, dim) = slots.shape[0], self._row
        shape = (layers, n, heads, dim)
        for name, t in (("k", k), ("v", v)):
            if t.shape != shape or t.dtype is not k.dtype or (n and t.stride(3) != 1):
                raise ValueError(f"{name}: expects {shape} of one type, head_dim contiguous; got "
                                 f"{tuple(t.shape)} {t.dtype}")
        return _ROWS.pack(self._dtype("k", k), 0, n, k.data_ptr(), v.data_ptr(), *_strides(k),
                          *_strides(v), slots.data_ptr())

    def write(self, k, v, slots, stream=None):
        """Quantises tokens' k and v ([layers, tokens, kv_heads, head_dim], bf16 or
        fp16, any strides that are multiples of 8) into ``slots`` (device int64, each
        named once; negative: skipped)."""
        s = self._here(stream, k, v, slots)
        st = self._write(self._desc, self._rows(k, v, slots), self._status, s)
        if st:
            raise KvcError(st, "kvc_cache_write")

    def read(self, slots, k=None, v=None, dtype=None, stream=None):
        """The rows stored in ``slots``, into k and v (made here if not given, with
        zeros for negative slots; rows of given tensors are left as they were)."""
        import torch
        if (k is None) != (v is None):
            raise ValueError("give both k and v, or neither")
        s = self._here(stream, k, v, slots)
        if k is None:
            d = self.desc
            with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
                k, v = (torch.zeros(d.layers, slots.numel(), d.kv_heads, d.head_dim,
                                    dtype=dtype or torch.bfloat16, device=self.device)
                        for _ in range(2))
        st = self._read(self._desc, self._rows(k, v, slots), self._status, s)
        if st:
            raise KvcError(st, "kvc_cache_read")
        return k, v

    def load(self, stream_buf, nbytes: int, slots, seq_lens, stream=None, check: bool = False):
        """Puts a compressed stream's codes into ``slots`` (one per token, requests in
        order). An error in the stream or the slots goes to the status word that ``check``
        reads; with check=True (which waits for the load) it raises here instead."""
        import torch
        if slots.dtype is not torch.int64 or slots.dim() != 1 or not slots.is_contiguous():
            raise ValueError("slots: expects a contiguous int64 vector")
        if slots.shape[0] != sum(seq_lens):
            raise ValueError(f"{slots.shape[0]} slots for {sum(seq_lens)} tokens")
        if stream_buf.dtype != torch.uint8 or not 0 <= int(nbytes) <= stream_buf.numel() or \
                not stream_buf.is_contiguous():
            raise ValueError("stream_buf: expects a contiguous uint8 buffer of nbytes")
        s = self._here(stream, stream_buf, slots)
        if check:
            self._may_wait(stream, "load(check=True)")
        n = len(seq_lens)
        seq, L, D = (C.c_int32 * (n or 1))(*map(int, seq_lens)), lib(), C.byref(self.desc)
        self._with_workspace(
            "kvc_cache_load", stream, s, lambda: L.kvc_cache_load_workspace_bytes(D, seq, n),
            lambda at, size: L.kvc_cache_load_noting(stream_buf.data_ptr(), int(nbytes), D, seq, n,
                                                     slots.data_ptr(), at, size,
                                                     None if check else self._status, s),
            (lambda at: kvc_stream_status(at, s)) if check else None)

    def attend(self, q, page_table, seq_lens, q_starts=None, max_q: int = 1, out=None, lse=None,
               scale: float | None = None, causal: bool = True, window: int = 0, stream=None):
        """Attention of q ([layers, rows, heads, head_dim], bf16 or fp16) over the
        requests' pages: page_table int32 [n_requests, pages], seq_lens int32
        [n_requests] (the query tokens' own keys among them), q_starts int32
        [n_requests + 1] (none: row r is request r's one query), all on the device;
        max_q: the most queries of one request. Returns out (made here with zeros
        if not given); lse, if given, is fp32 [layers, rows, heads]."""
        import torch
        (layers, heads, dim), int32 = self._row, torch.int32
        s = self._here(stream, q, page_table, seq_lens, q_starts, out, lse)
        n, shape, heads = seq_lens.numel(), q.shape, heads or 1
        if len(shape) != 4 or shape[0] != layers or shape[3] != dim or shape[2] % heads or \
                (shape[1] and q.stride(3) != 1):
            raise ValueError(f"q: expects [{layers}, rows, a multiple of {heads}, {dim}]")
        if page_table.dtype is not int32 or page_table.dim() != 2 or page_table.shape[0] != n or \
                (page_table.numel() and page_table.stride(1) != 1):
            raise ValueError(f"page_table: expects int32 [{n}, pages]")
        if seq_lens.dtype is not int32 or seq_lens.dim() != 1 or (n > 1 and seq_lens.stride(0) != 1):
            raise ValueError("seq_lens: expects an int32 vector")
        if q_starts is not None and (q_starts.dtype is not int32 or q_starts.shape != (n + 1,) or
                                     not q_starts.is_contiguous()):
            raise ValueError(f"q_starts: expects int32 [{n + 1}]")
        if out is None:
            with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
                out = torch.zeros(shape, dtype=q.dtype, device=self.device)
        elif out.shape != shape or out.dtype is not q.dtype or (shape[1] and out.stride(3) != 1):
            raise ValueError("out: expects the shape and type of q")
        if lse is not None and (lse.dtype is not torch.float32 or lse.shape != shape[:3] or
                                not lse.is_contiguous()):
            raise ValueError("lse: expects contiguous float32 [layers, rows, heads]")
        try:
            t = _ATTN.pack(self._dtype("q", q), shape[2] // heads, n, max_q, 1 if causal else 0, window,
                           dim ** -0.5 if scale is None else scale, 0, shape[1],
                           0 if q_starts is None else q_starts.data_ptr(), seq_lens.data_ptr(),
                           page_table.data_ptr(), page_table.shape[1],
                           page_table.stride(0) if n > 1 else 0, q.data_ptr(), *_strides(q),
                           out.data_ptr(), *_strides(out), 0 if lse is None else lse.data_ptr())
        except (struct.error, OverflowError) as e:
            raise ValueError(f"max_q, window, scale: {e}") from None
        self._with_workspace(
            "kvc_cache_attend", stream, s, lambda: lib().kvc_cache_attend_workspace_bytes(
                C.byref(self.desc), C.cast(t, C.POINTER(kvc_cache_attn))),
            lambda at, size: self._attend(self._desc, t, at, size, self._status, s))
        return out

    def check(self, stream=None):
        """Waits for the stream, raises the first data-dependent error since the last
        check, and clears it."""
        s = self._here(stream)
        self._may_wait(stream, "check()")
        st = kvc_stream_status(self._status, s)
        if st != KVC_OK:
            kvc_cache_status_clear(self._status, s)
            raise KvcError(st, "PagedCache (device)")
