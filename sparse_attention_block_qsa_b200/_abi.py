"""ctypes binding of ``libqsa.so`` (the C ABI declared in include/qsa.h).

Argument marshalling only: torch tensors supply device pointers, strides and
the current stream; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the library or a GPU is missing the
calls raise.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqsa.so")
SCALE = 1.0 / math.sqrt(128.0)

_i64, _i32, _f32, _vp, _sz = C.c_int64, C.c_int32, C.c_float, C.c_void_p, C.c_size_t

# the 8-bit cache: codes, scales and their strides, then the page table
_CACHE8 = [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64, _i64, _i64, _i64, _i64, _i32, _vp, _i64, _i32, _vp, _vp, _i32]
_APPEND = [_vp, _i64, _i64, _vp, _i64, _i64, *_CACHE8, _i64, _vp, _vp]
_ATTN8 = [_vp, _i64, _i64, _i32, *_CACHE8, _vp, _i64, _i32, _i64, _vp, _f32, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp]

SIGNATURES = {
    "qsa_status_string": (C.c_char_p, [C.c_int]),
    "qsa_last_error_detail": (C.c_char_p, []),
    "qsa_device_error": (C.c_int, [C.POINTER(C.c_uint32)]),
    "qsa_selftest_bounded_wait": (C.c_int, [C.c_uint64, _i32, _vp]),
    "qsa_mqa_decode": (C.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i32, _i64, _i64, _vp, _i64, _i32,
                                 _vp, _i32, _i32, _f32, _vp, _i64, _i64, _i32, _vp]),
    "qsa_mqa_decode_f16": (C.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i32, _i64, _i64, _vp, _i64, _i32,
                                     _vp, _i32, _i32, _f32, _vp, _i64, _i64, _i32, _vp]),
    "qsa_mqa_prefill_f16": (C.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _f32, _vp, _i64,
                                      _i32, _vp]),
    "qsa_mqa_decode_fp8": (C.c_int, [_vp, _i64, _i64, _i64, _vp, _f32, _i64, _i32, _i64, _i64, _vp, _i64,
                                     _i32, _vp, _i32, _i32, _f32, _vp, _i64, _i64, _i32, _vp]),
    "qsa_mqa_prefill": (C.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _f32, _vp, _i64,
                                  _i32, _vp]),
    "qsa_prefill_intervals": (C.c_int, [_vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp]),
    "qsa_topk": (C.c_int, [_vp, _i64, _vp, _i64, _i32, _i32, _vp, _i64, _vp]),
    "qsa_topk_ws": (C.c_int, [_vp, _i64, _vp, _i64, _i32, _i32, _vp, _i64, _vp, C.c_size_t, _vp]),
    "qsa_topk_workspace_size": (C.c_size_t, [_i64, _i32, _i32]),
    "qsa_mqa_prefill_topk": (C.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _f32, _i32,
                                       _i32, _vp, _i64, _vp, _sz, _vp]),
    "qsa_prefill_topk_workspace_size": (_sz, [_i64, _i32]),
    "qsa_mqa_prefill_topk_noalloc": (C.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _f32, _i32,
                                               _i32, _vp, _i64, _vp]),
    "qsa_expand_block_indices": (C.c_int, [_vp, _i64, _i32, _vp, _vp, _i32, _i64, _vp, _i64, _vp]),
    "qsa_sparse_attention": (C.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _i64, _i32, _i64, _i64, _i64, _i32,
                                       _vp, _i64, _i32, _vp, _vp, _i32, _vp, _i64, _i32, _i64, _vp, _f32,
                                       _vp, _i64, _vp, _vp, _sz, _vp]),
    "qsa_sparse_attention_workspace_size": (_sz, [_i64, _i32, _i32, _i32]),
    "qsa_mqa_paged_batch": (C.c_int, [_vp, _i64, _i64, _vp, _i64, _i32, _i64, _i64, _vp, _i64, _i32, _vp, _vp,
                                      _i32, _i32, _i32, _i64, _f32, _vp, _i64, _i32, _vp, _sz, _vp]),
    "qsa_mqa_paged_batch_workspace_size": (_sz, [_i32, _i32, _i32, _i64, _i32]),
    "qsa_kv_append_fp8": (C.c_int, _APPEND),
    "qsa_kv_append_fp8_f16": (C.c_int, _APPEND),
    "qsa_sparse_attention_fp8": (C.c_int, _ATTN8),
    "qsa_sparse_attention_fp8_f16": (C.c_int, _ATTN8),
    "qsa_sparse_attention_fp8_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "qsa_accumulate_weights": (C.c_int, [_vp, _i64, _vp, _i64, _i32, _i64, _vp, _i64, _i32, _vp, _vp, _i32, _vp,
                                         _i64, _i32, _vp]),
    "qsa_evict_pages": (C.c_int, [_vp, _i64, _i32, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _i64, _vp,
                                  _i64, _vp, _vp, _sz, _vp]),
    "qsa_evict_pages_workspace_size": (_sz, [_i32, _i32, _i32]),
}

STATUS = {0: "QSA_OK", 1: "QSA_ERR_INVALID_ARG", 2: "QSA_ERR_ALIGNMENT", 3: "QSA_ERR_UNSUPPORTED",
          4: "QSA_ERR_WORKSPACE", 5: "QSA_ERR_CUDA"}


class QSAError(RuntimeError):
    def __init__(self, call: str, status: int, detail: str):
        self.call, self.status, self.detail = call, status, detail
        super().__init__(f"{call}: {STATUS.get(status, status)}: {detail}")


_lib = None


def lib() -> C.CDLL:
    """Load the in-tree library (built by ``python -m sparse_attention_block_qsa_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m sparse_attention_block_qsa_b200.build`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _check(call: str, status: int) -> None:
    if status != 0:
        raise QSAError(call, status, lib().qsa_last_error_detail().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, dim: int) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")


def device_error() -> int:
    """Read and clear the library's device error word (synchronises)."""
    v = C.c_uint32(0)
    _check("qsa_device_error", lib().qsa_device_error(C.byref(v)))
    return v.value


def selftest_bounded_wait(timeout_ns: int, arrive: bool, stream=None) -> None:
    """Launch the bounded-wait diagnostic (a wait on a barrier phase that
    nothing completes unless `arrive`); see qsa_selftest_bounded_wait."""
    _check("qsa_selftest_bounded_wait", lib().qsa_selftest_bounded_wait(timeout_ns, 1 if arrive else 0,
                                                                       _stream(stream)))


def _decode_checks(q, k_cache, page_table, seq_lens, W, out, q_dtype=torch.bfloat16):
    _need(q, "q", q_dtype, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, Q = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((B, Q, W), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, 3)
    if q.shape[2:] != (4, 128) or q.stride(3) != 1:
        raise ValueError("q must be [B, Q, 4, 128] with unit feature stride")
    if k_cache.shape[2:] != (1, 128) or k_cache.stride(3) != 1:
        raise ValueError("k_cache must be [pages, page_size, 1, 128] with unit feature stride")
    if page_table.stride(1) != 1 or seq_lens.stride(0) != 1 or out.stride(2) != 1:
        raise ValueError("page_table, seq_lens and out need a unit innermost stride")
    if out.shape[:2] != (B, Q) or page_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("batch shapes of q, page_table, seq_lens and out disagree")
    return B, Q, out


def mqa_decode(q: torch.Tensor, k_cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
               W: int, scale: float = SCALE, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode / spec-decode scores: q [B, Q, 4, 128] and k_cache [pages,
    page_size, 1, 128] both bf16 or both fp16, page_table int32 [B,
    max_pages], seq_lens int32 [B] (tokens) -> out fp32 [B, Q, W]."""
    dt = q.dtype if isinstance(q, torch.Tensor) and q.dtype == torch.float16 else torch.bfloat16
    _need(k_cache, "k_cache", dt, 4)
    B, Q, out = _decode_checks(q, k_cache, page_table, seq_lens, W, out, dt)
    name = "qsa_mqa_decode_f16" if dt == torch.float16 else "qsa_mqa_decode"
    _check(name, getattr(lib(), name)(
        _ptr(q), q.stride(0), q.stride(1), q.stride(2),
        _ptr(k_cache), k_cache.shape[0], k_cache.shape[1], k_cache.stride(0), k_cache.stride(1),
        _ptr(page_table), page_table.stride(0), page_table.shape[1], _ptr(seq_lens), B, Q, scale,
        _ptr(out), out.stride(0), out.stride(1), out.shape[2], _stream(stream)))
    return out


def mqa_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, k_scale: float, page_table: torch.Tensor,
                   seq_lens: torch.Tensor, W: int, scale: float = SCALE, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """mqa_decode over an fp8 E4M3 key cache: k_cache float8_e4m3fn (or uint8
    codes) [pages, page_size, 1, 128] holding e4m3(bf16(k) / k_scale); keys
    are read as E4M3 value * k_scale (k_scale > 0)."""
    if isinstance(k_cache, torch.Tensor) and k_cache.dtype == torch.float8_e4m3fn:
        k_cache = k_cache.view(torch.uint8)
    _need(k_cache, "k_cache", torch.uint8, 4)
    B, Q, out = _decode_checks(q, k_cache, page_table, seq_lens, W, out)
    _check("qsa_mqa_decode_fp8", lib().qsa_mqa_decode_fp8(
        _ptr(q), q.stride(0), q.stride(1), q.stride(2),
        _ptr(k_cache), float(k_scale), k_cache.shape[0], k_cache.shape[1], k_cache.stride(0), k_cache.stride(1),
        _ptr(page_table), page_table.stride(0), page_table.shape[1], _ptr(seq_lens), B, Q, scale,
        _ptr(out), out.stride(0), out.stride(1), out.shape[2], _stream(stream)))
    return out


def _prefill_checks(q, k, ks, ke, dt=torch.bfloat16):
    _need(q, "q", dt, 3)
    _need(k, "k", dt, 2)
    _need(ks, "ks", torch.int32, 1)
    _need(ke, "ke", torch.int32, 1)
    if q.shape[1:] != (4, 128) or q.stride(2) != 1:
        raise ValueError("q must be [T, 4, 128] with unit feature stride")
    if k.shape[1] != 128 or k.stride(1) != 1:
        raise ValueError("k must be [Nk, 128] with unit feature stride")
    if ks.shape[0] != q.shape[0] or ke.shape[0] != q.shape[0] or ks.stride(0) != 1 or ke.stride(0) != 1:
        raise ValueError("ks and ke must be contiguous int32 [T]")


def mqa_prefill(q: torch.Tensor, k: torch.Tensor, ks: torch.Tensor, ke: torch.Tensor, W: int,
                scale: float = SCALE, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prefill scores: q [T, 4, 128] and k [Nk, 128] both bf16 or both fp16,
    ks/ke int32 [T] -> out fp32 [T, W] with out[t, j] the score of key ks[t] + j."""
    dt = q.dtype if isinstance(q, torch.Tensor) and q.dtype == torch.float16 else torch.bfloat16
    _prefill_checks(q, k, ks, ke, dt)
    T = q.shape[0]
    if out is None:
        out = torch.empty((T, W), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, 2)
    if out.shape[0] != T or out.stride(1) != 1:
        raise ValueError("out must be [T, W] with unit column stride")
    name = "qsa_mqa_prefill_f16" if dt == torch.float16 else "qsa_mqa_prefill"
    _check(name, getattr(lib(), name)(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0), k.shape[0], _ptr(ks), _ptr(ke), T, scale,
        _ptr(out), out.stride(0), out.shape[1], _stream(stream)))
    return out


def prefill_intervals(cu_seqlens_q: torch.Tensor, seq_lens: torch.Tensor, key_offsets: torch.Tensor, T: int,
                      ks: torch.Tensor | None = None, ke: torch.Tensor | None = None, stream=None):
    """Per-row key intervals (ks, ke) int32 [T] of a packed prefill batch."""
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (seq_lens, "seq_lens"), (key_offsets, "key_offsets")):
        _need(t, n, torch.int32, 1)
        if t.stride(0) != 1:
            raise ValueError(f"{n} must be contiguous")
    S = seq_lens.shape[0]
    if cu_seqlens_q.shape[0] != S + 1 or key_offsets.shape[0] != S:
        raise ValueError("cu_seqlens_q must have S + 1 entries and key_offsets S")
    dev = seq_lens.device
    ks = torch.empty(T, dtype=torch.int32, device=dev) if ks is None else ks
    ke = torch.empty(T, dtype=torch.int32, device=dev) if ke is None else ke
    _check("qsa_prefill_intervals", lib().qsa_prefill_intervals(
        _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(key_offsets), S, T, _ptr(ks), _ptr(ke), _stream(stream)))
    return ks, ke


def topk_workspace_size(rows: int, W: int, k: int) -> int:
    return int(lib().qsa_topk_workspace_size(rows, W, k))


def topk(scores: torch.Tensor, k: int, lengths: torch.Tensor | None = None, idx: torch.Tensor | None = None,
         stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Top-k column indices int32 [rows, k] (ascending, -1 padded) of score rows fp32 [rows, W];
    with a workspace (a device tensor of at least topk_workspace_size bytes) through qsa_topk_ws."""
    _need(scores, "scores", torch.float32, 2)
    if scores.stride(1) != 1:
        raise ValueError("scores need a unit column stride")
    rows, W = scores.shape
    if lengths is not None:
        _need(lengths, "lengths", torch.int32, 1)
        if lengths.shape[0] != rows or lengths.stride(0) != 1:
            raise ValueError("lengths must be contiguous int32 [rows]")
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=scores.device)
    _need(idx, "idx", torch.int32, 2)
    if idx.shape != (rows, k) or idx.stride(1) != 1:
        raise ValueError("idx must be [rows, k] with unit column stride")
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        nbytes = workspace.numel() * workspace.element_size()
        _check("qsa_topk_ws", lib().qsa_topk_ws(_ptr(scores), scores.stride(0), _ptr(lengths), rows, W, k, _ptr(idx),
                                                idx.stride(0), _ptr(workspace), nbytes, _stream(stream)))
        return idx
    _check("qsa_topk", lib().qsa_topk(_ptr(scores), scores.stride(0), _ptr(lengths), rows, W, k, _ptr(idx),
                                      idx.stride(0), _stream(stream)))
    return idx


def prefill_topk_workspace_size(T: int, W: int) -> int:
    return int(lib().qsa_prefill_topk_workspace_size(T, W))


def mqa_prefill_topk(q: torch.Tensor, k: torch.Tensor, ks: torch.Tensor, ke: torch.Tensor, W: int,
                     topk_k: int, workspace: torch.Tensor, scale: float = SCALE,
                     idx: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prefill scores followed by per-row top-k, chunked through ``workspace``
    (a CUDA tensor, any dtype, 16-byte aligned) -> idx int32 [T, topk_k]."""
    _prefill_checks(q, k, ks, ke)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    T = q.shape[0]
    if idx is None:
        idx = torch.empty((T, topk_k), dtype=torch.int32, device=q.device)
    _need(idx, "idx", torch.int32, 2)
    if idx.shape != (T, topk_k) or idx.stride(1) != 1:
        raise ValueError("idx must be [T, topk_k] with unit column stride")
    _check("qsa_mqa_prefill_topk", lib().qsa_mqa_prefill_topk(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0), k.shape[0], _ptr(ks), _ptr(ke), T, scale, W,
        topk_k, _ptr(idx), idx.stride(0), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return idx


def mqa_prefill_topk_noalloc(q: torch.Tensor, k: torch.Tensor, ks: torch.Tensor, ke: torch.Tensor, W: int,
                             topk_k: int, scale: float = SCALE, idx: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """Prefill scores followed by per-row top-k through the library's static
    scratch (no device allocation by the library) -> idx int32 [T, topk_k].
    Calls that overlap on the GPU share that scratch and must be serialised."""
    _prefill_checks(q, k, ks, ke)
    T = q.shape[0]
    if idx is None:
        idx = torch.empty((T, topk_k), dtype=torch.int32, device=q.device)
    _need(idx, "idx", torch.int32, 2)
    if idx.shape != (T, topk_k) or idx.stride(1) != 1:
        raise ValueError("idx must be [T, topk_k] with unit column stride")
    _check("qsa_mqa_prefill_topk_noalloc", lib().qsa_mqa_prefill_topk_noalloc(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0), k.shape[0], _ptr(ks), _ptr(ke), T, scale, W,
        topk_k, _ptr(idx), idx.stride(0), _stream(stream)))
    return idx


def _index_checks(cu_seqlens_q, seq_lens):
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (seq_lens, "seq_lens")):
        _need(t, n, torch.int32, 1)
        if t.stride(0) != 1:
            raise ValueError(f"{n} must be contiguous")
    if cu_seqlens_q.shape[0] != seq_lens.shape[0] + 1:
        raise ValueError("cu_seqlens_q must have one more entry than seq_lens")


def expand_block_indices(blocks: torch.Tensor, cu_seqlens_q: torch.Tensor, seq_lens: torch.Tensor,
                         token_idx: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Selected blocks int32 [T, k] -> token indices int32 [T, 4k + 3] (four
    tokens per block, then the row's open group, then -1)."""
    _need(blocks, "blocks", torch.int32, 2)
    _index_checks(cu_seqlens_q, seq_lens)
    if blocks.stride(1) != 1:
        raise ValueError("blocks need a unit column stride")
    T, k = blocks.shape
    if token_idx is None:
        token_idx = torch.empty((T, 4 * k + 3), dtype=torch.int32, device=blocks.device)
    _need(token_idx, "token_idx", torch.int32, 2)
    if token_idx.shape != (T, 4 * k + 3) or token_idx.stride(1) != 1:
        raise ValueError("token_idx must be [T, 4k + 3] with unit column stride")
    _check("qsa_expand_block_indices", lib().qsa_expand_block_indices(
        _ptr(blocks), blocks.stride(0), k, _ptr(cu_seqlens_q), _ptr(seq_lens), seq_lens.shape[0], T,
        _ptr(token_idx), token_idx.stride(0), _stream(stream)))
    return token_idx


def sparse_attention_workspace_size(T: int, Hq: int, Hkv: int, width: int) -> int:
    return int(lib().qsa_sparse_attention_workspace_size(T, Hq, Hkv, width))


def sparse_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                     cu_seqlens_q: torch.Tensor, seq_lens: torch.Tensor, token_idx: torch.Tensor, scale: float,
                     gate: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Sparse core attention: q bf16 [T, Hq, 256], K/V bf16 [pages, page_size,
    Hkv, 256], token_idx int32 [T, width] -> (out bf16 [T, Hq, 256], lse fp32
    [T, Hq]).  The workspace (any CUDA tensor, 16-byte aligned) is allocated
    here by torch when not given."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(token_idx, "token_idx", torch.int32, 2)
    _index_checks(cu_seqlens_q, seq_lens)
    T, Hq, Dq = q.shape
    if Dq != 256 or q.stride(2) != 1:
        raise ValueError("q must be [T, Hq, 256] with unit feature stride")
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride() or k_cache.shape[3] != 256 \
            or k_cache.stride(3) != 1:
        raise ValueError("k_cache and v_cache must be [pages, page_size, Hkv, 256] with the same strides")
    if token_idx.shape[0] != T or token_idx.stride(1) != 1 or page_table.stride(1) != 1:
        raise ValueError("token_idx must be [T, width] and page_table [R, max_pages], unit column strides")
    if page_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("page_table needs one row per request")
    Hkv = k_cache.shape[2]
    width = token_idx.shape[1]
    if gate is not None:
        _need(gate, "gate", torch.float32, 2)
        if gate.shape != (T, Hq) or not gate.is_contiguous():
            raise ValueError("gate must be contiguous fp32 [T, Hq]")
    if out is None:
        out = torch.empty((T, Hq, 256), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    if out.shape != (T, Hq, 256) or out.stride(2) != 1 or out.stride(1) != 256:
        raise ValueError("out must be [T, Hq, 256] with contiguous heads")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    _need(lse, "lse", torch.float32, 2)
    if lse.shape != (T, Hq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [T, Hq]")
    need = sparse_attention_workspace_size(T, Hq, Hkv, max(width, 1))
    if workspace is None:
        workspace = torch.empty(max(need, 16) // 4 + 4, dtype=torch.float32, device=q.device)
    _check("qsa_sparse_attention", lib().qsa_sparse_attention(
        _ptr(q), q.stride(0), q.stride(1), Hq, _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], k_cache.shape[1],
        k_cache.stride(0), k_cache.stride(1), k_cache.stride(2), Hkv, _ptr(page_table), page_table.stride(0),
        page_table.shape[1], _ptr(cu_seqlens_q), _ptr(seq_lens), seq_lens.shape[0], _ptr(token_idx),
        token_idx.stride(0), width, T, _ptr(gate), float(scale), _ptr(out), out.stride(0), _ptr(lse),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return out, lse


def paged_batch_workspace_size(R: int, num_decodes: int, decode_query_len: int, T: int, W: int) -> int:
    return int(lib().qsa_mqa_paged_batch_workspace_size(R, num_decodes, decode_query_len, T, W))


def mqa_paged_batch(q: torch.Tensor, k_cache: torch.Tensor, page_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    seq_lens: torch.Tensor, num_decodes: int, decode_query_len: int, W: int, scale: float = SCALE,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Scores of a mixed batch from the paged cache: q bf16 [T, 4, 128] (the
    num_decodes x decode_query_len decode rows first), k_cache bf16 [pages,
    page_size, 1, 128], page_table int32 [R, max_pages], cu_seqlens_q int32
    [R + 1], seq_lens int32 [R] -> out fp32 [T, W] (request-local key
    columns).  The workspace is allocated here by torch when not given."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _index_checks(cu_seqlens_q, seq_lens)
    if q.shape[1:] != (4, 128) or q.stride(2) != 1:
        raise ValueError("q must be [T, 4, 128] with unit feature stride")
    if k_cache.shape[2:] != (1, 128) or k_cache.stride(3) != 1 or page_table.stride(1) != 1:
        raise ValueError("k_cache must be [pages, page_size, 1, 128]; page_table needs a unit column stride")
    T = q.shape[0]
    R = seq_lens.shape[0]
    if out is None:
        out = torch.empty((T, W), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, 2)
    if out.shape != (T, W) or out.stride(1) != 1:
        raise ValueError("out must be [T, W] with unit column stride")
    if workspace is None:
        need = paged_batch_workspace_size(R, num_decodes, decode_query_len, T, W)
        workspace = torch.empty(max(need, 16) // 4 + 4, dtype=torch.float32, device=q.device)
    _check("qsa_mqa_paged_batch", lib().qsa_mqa_paged_batch(
        _ptr(q), q.stride(0), q.stride(1), _ptr(k_cache), k_cache.shape[0], k_cache.shape[1], k_cache.stride(0),
        k_cache.stride(1), _ptr(page_table), page_table.stride(0), page_table.shape[1], _ptr(cu_seqlens_q),
        _ptr(seq_lens), R, num_decodes, decode_query_len, T, scale, _ptr(out), out.stride(0), W,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


# The calls on the 8-bit cache are short on the device, so their binding keeps the host's share small: plain integers
# for pointers, every tensor's shape and strides read once, the checks in line.

def _fits(t, dtype, dim, dev):
    return t.dtype is dtype and t.get_device() == dev and t.dim() == dim


def _want(t, name, dtype, dim, dev):
    """_need, and that the tensor lives on device ordinal `dev`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or t.dim() != dim:
        _need(t, name, dtype, dim)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, other tensors on cuda:{dev}: one call needs one device")


def _first(t, name):
    """Device ordinal of a call's first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _raw_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(stream, shape, dtype, dev):
    """Memory that belongs to the stream the call runs on (an output or a workspace made here)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_raw_stream(stream, dev), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


_entries: dict = {}


def _call(dev, name, *args):
    """The library call with device `dev` current."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(lib(), name)
    if dev == torch._C._cuda_getDevice():
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status:
        _check(name, status)


def _workspace(workspace, need, stream, dev):
    """(pointer, bytes, the tensor that owns it)"""
    if workspace is None:
        if need <= 0:
            return 0, 0, None
        workspace = _new(stream, need, torch.uint8, dev)
        return workspace.data_ptr(), need, workspace
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if workspace.get_device() != dev:
        raise ValueError(f"workspace is on cuda:{workspace.get_device()}, other tensors on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


_CODES = (torch.float8_e4m3fn, torch.uint8)
_F32, _I32 = torch.float32, torch.int32


def _cache8(k_cache, v_cache, k_scale, v_scale, dev):
    """Check the 8-bit cache's tensors; returns (pages, page_size, Hkv, its C arguments from k_cache to Hkv)."""
    try:
        dt = k_cache.dtype
        ok = dt in _CODES and v_cache.dtype in _CODES and _fits(k_cache, dt, 4, dev) \
            and _fits(v_cache, v_cache.dtype, 4, dev) and _fits(k_scale, _F32, 3, dev) and _fits(v_scale, _F32, 3, dev)
    except AttributeError:
        ok = False
    if not ok:
        for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            if not isinstance(t, torch.Tensor) or t.dtype not in _CODES:
                _need(t, n, torch.uint8, 4)
            _want(t, n, t.dtype, 4, dev)
        _want(k_scale, "k_scale", torch.float32, 3, dev)
        _want(v_scale, "v_scale", torch.float32, 3, dev)
    shape, strides = k_cache.shape, k_cache.stride()
    pages, ps, Hkv, D = shape
    if v_cache.shape != shape or v_cache.stride() != strides or D != 256 or strides[3] != 1:
        raise ValueError("k_cache and v_cache must be [pages, page_size, Hkv, 256] with the same strides")
    sc_shape, sc_strides = k_scale.shape, k_scale.stride()
    blocks = sc_shape[1]
    if v_scale.shape != sc_shape or v_scale.stride() != sc_strides or sc_strides[2] != 1 or sc_shape[0] != pages \
            or sc_shape[2] != Hkv or blocks < 1 or ps % blocks:
        raise ValueError("k_scale and v_scale must be [pages, blocks, Hkv] with the same strides, unit head stride, "
                         "and blocks must divide page_size")
    return pages, ps, Hkv, (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, ps,
                            ps // blocks, strides[0], strides[1], strides[2], sc_strides[0], sc_strides[1], Hkv)


def _tables(page_table, cu_seqlens_q, seq_lens, dev):
    """Check the batch's tables; returns their C arguments from page_table to R."""
    try:
        ok = _fits(page_table, _I32, 2, dev) and _fits(cu_seqlens_q, _I32, 1, dev) and _fits(seq_lens, _I32, 1, dev)
    except AttributeError:
        ok = False
    if not ok:
        _want(page_table, "page_table", torch.int32, 2, dev)
        _want(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
        _want(seq_lens, "seq_lens", torch.int32, 1, dev)
    R, max_pages = page_table.shape
    pt_strides = page_table.stride()
    if seq_lens.shape[0] != R or pt_strides[1] != 1:
        raise ValueError("page_table needs one row per request and a unit column stride")
    if cu_seqlens_q.shape[0] != R + 1 or not cu_seqlens_q.is_contiguous() or not seq_lens.is_contiguous():
        raise ValueError("cu_seqlens_q must have one more entry than seq_lens, both contiguous")
    return page_table.data_ptr(), pt_strides[0], max_pages, cu_seqlens_q.data_ptr(), seq_lens.data_ptr(), R


def _token_weight(token_weight, pages, page_size, dev):
    _want(token_weight, "token_weight", torch.int64, 2, dev)
    if token_weight.shape != (pages, page_size) or not token_weight.is_contiguous():
        raise ValueError("token_weight must be contiguous int64 [pages, page_size]")


def kv_append_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  k_scale: torch.Tensor, v_scale: torch.Tensor, page_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                  seq_lens: torch.Tensor, token_weight: torch.Tensor | None = None, stream=None) -> None:
    """Quantise new rows k, v (bf16 or fp16 [T, Hkv, 256]) into the 8-bit cache, in place: k_cache, v_cache
    float8_e4m3fn (or uint8 codes) [pages, page_size, Hkv, 256], k_scale, v_scale fp32 [pages, page_size /
    block_tokens, Hkv].  Row i of request r goes to position seq_lens[r] - qlen_r + i.  A block's scale is the
    smallest power of two that holds it; it grows when a later token needs it.  token_weight (int64 [pages,
    page_size]) is zeroed for the tokens written."""
    dev = _first(k, "k")
    dt = torch.float16 if k.dtype == torch.float16 else torch.bfloat16
    _want(k, "k", dt, 3, dev)
    _want(v, "v", dt, 3, dev)
    pages, ps, Hkv, cache = _cache8(k_cache, v_cache, k_scale, v_scale, dev)
    tables = _tables(page_table, cu_seqlens_q, seq_lens, dev)
    shape, ks, vs = k.shape, k.stride(), v.stride()
    T = shape[0]
    if v.shape != shape or shape[1] != Hkv or shape[2] != 256 or ks[2] != 1 or vs[2] != 1:
        raise ValueError("k and v must be [T, Hkv, 256] with unit feature stride")
    if token_weight is not None:
        _token_weight(token_weight, pages, ps, dev)
    _call(dev, "qsa_kv_append_fp8_f16" if dt == torch.float16 else "qsa_kv_append_fp8", k.data_ptr(), ks[0], ks[1],
          v.data_ptr(), vs[0], vs[1], *cache, *tables, T, None if token_weight is None else token_weight.data_ptr(),
          _raw_stream(stream, dev))


@functools.lru_cache(maxsize=1024)
def sparse_attention_fp8_workspace_size(T: int, Hq: int, Hkv: int, width: int, weights: bool = False) -> int:
    return int(lib().qsa_sparse_attention_fp8_workspace_size(T, Hq, Hkv, width, 1 if weights else 0))


def sparse_attention_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, page_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                         seq_lens: torch.Tensor, token_idx: torch.Tensor, scale: float,
                         gate: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         lse: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None):
    """sparse_attention over the 8-bit cache of kv_append_fp8: q bf16 or fp16 [T, Hq, 256] -> (out of q's type
    [T, Hq, 256], lse fp32 [T, Hq]).  weights (fp32 [T, width]), if given, receives every entry's softmax
    probability summed over the query heads.  The workspace (any CUDA tensor, 16-byte aligned) is allocated here by
    torch when not given."""
    dev = _first(q, "q")
    dt = torch.float16 if q.dtype == torch.float16 else torch.bfloat16
    _want(q, "q", dt, 3, dev)
    pages, ps, Hkv, cache = _cache8(k_cache, v_cache, k_scale, v_scale, dev)
    tables = _tables(page_table, cu_seqlens_q, seq_lens, dev)
    _want(token_idx, "token_idx", torch.int32, 2, dev)
    T, Hq, Dq = q.shape
    qs, ts = q.stride(), token_idx.stride()
    rows, width = token_idx.shape
    if Dq != 256 or qs[2] != 1:
        raise ValueError("q must be [T, Hq, 256] with unit feature stride")
    if rows != T or ts[1] != 1:
        raise ValueError("token_idx must be [T, width] with unit column stride")
    gate_p = weights_p = None
    ws0 = 0
    if gate is not None:
        _want(gate, "gate", torch.float32, 2, dev)
        if gate.shape != (T, Hq) or not gate.is_contiguous():
            raise ValueError("gate must be contiguous fp32 [T, Hq]")
        gate_p = gate.data_ptr()
    if weights is not None:
        _want(weights, "weights", torch.float32, 2, dev)
        ws0, ws1 = weights.stride()
        if weights.shape != (T, width) or ws1 != 1:
            raise ValueError("weights must be fp32 [T, width] with unit column stride")
        weights_p = weights.data_ptr()
    if out is None:
        out = torch.empty_like(q) if stream is None and q.is_contiguous() else _new(stream, (T, Hq, 256), dt, dev)
        out0 = Hq * 256
    else:
        _want(out, "out", dt, 3, dev)
        out0, out1, out2 = out.stride()
        if out.shape != (T, Hq, 256) or out2 != 1 or out1 != 256:
            raise ValueError("out must be [T, Hq, 256] with contiguous heads")
    if lse is None:
        lse = _new(stream, (T, Hq), torch.float32, dev)
    else:
        _want(lse, "lse", torch.float32, 2, dev)
        if lse.shape != (T, Hq) or not lse.is_contiguous():
            raise ValueError("lse must be contiguous fp32 [T, Hq]")
    need = 0
    if workspace is None:
        need = sparse_attention_fp8_workspace_size(T, Hq, Hkv, width, weights is not None)
    wp, nbytes, workspace = _workspace(workspace, need, stream, dev)
    _call(dev, "qsa_sparse_attention_fp8_f16" if dt == torch.float16 else "qsa_sparse_attention_fp8",
          q.data_ptr(), qs[0], qs[1], Hq, *cache, *tables, token_idx.data_ptr(), ts[0], width, T, gate_p, scale,
          out.data_ptr(), out0, lse.data_ptr(), weights_p, ws0, wp, nbytes, _raw_stream(stream, dev))
    return out, lse


def accumulate_weights(weights: torch.Tensor, token_idx: torch.Tensor, page_table: torch.Tensor,
                       cu_seqlens_q: torch.Tensor, seq_lens: torch.Tensor, token_weight: torch.Tensor,
                       stream=None) -> torch.Tensor:
    """Add attention weights (fp32 [T, width], one per entry of token_idx int32 [T, width]) up per cached token, in
    place: token_weight int64 [pages, page_size] in units of 2^-32.  Returns token_weight."""
    dev = _first(weights, "weights")
    _want(weights, "weights", torch.float32, 2, dev)
    _want(token_idx, "token_idx", torch.int32, 2, dev)
    _want(token_weight, "token_weight", torch.int64, 2, dev)
    tables = _tables(page_table, cu_seqlens_q, seq_lens, dev)
    pages, ps = token_weight.shape
    T, width = shape = token_idx.shape
    ws, ts = weights.stride(), token_idx.stride()
    if not token_weight.is_contiguous():
        raise ValueError("token_weight must be contiguous int64 [pages, page_size]")
    if weights.shape != shape or ws[1] != 1 or ts[1] != 1:
        raise ValueError("weights and token_idx must be [T, width] with unit column strides")
    _call(dev, "qsa_accumulate_weights", weights.data_ptr(), ws[0], token_idx.data_ptr(), ts[0], width, T, *tables,
          token_weight.data_ptr(), pages, ps, _raw_stream(stream, dev))
    return token_weight


@functools.lru_cache(maxsize=1024)
def evict_pages_workspace_size(R: int, max_pages: int, page_size: int) -> int:
    return int(lib().qsa_evict_pages_workspace_size(R, max_pages, page_size))


def evict_pages(token_weight: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, keep: torch.Tensor,
                keep_first: int = 0, keep_last: int = 1, table_out: torch.Tensor | None = None,
                freed: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """Drop the pages of least accumulated weight (token_weight int64 [pages, page_size]) until request r has
    keep[r] (int32 [R]) live pages; its first keep_first and last keep_last logical pages stay.  Returns (table_out
    int32 [R, max_pages] with -1 for dropped pages, freed int32 [R, max_pages]: the dropped pages in order, then -1,
    counts int32 [R]).  table_out may be page_table."""
    dev = _first(token_weight, "token_weight")
    _want(token_weight, "token_weight", torch.int64, 2, dev)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(seq_lens, "seq_lens", torch.int32, 1, dev)
    _want(keep, "keep", torch.int32, 1, dev)
    pages, ps = token_weight.shape
    R, max_pages = shape = page_table.shape
    pts = page_table.stride()
    if not token_weight.is_contiguous():
        raise ValueError("token_weight must be contiguous int64 [pages, page_size]")
    if seq_lens.shape[0] != R or keep.shape[0] != R or not seq_lens.is_contiguous() or not keep.is_contiguous() \
            or pts[1] != 1:
        raise ValueError("page_table needs one row per request and a unit column stride, seq_lens and keep one "
                         "contiguous entry per request")
    if table_out is None and freed is None:
        table_out, freed = _new(stream, (2, R, max_pages), torch.int32, dev).unbind(0)
        out0 = freed0 = max_pages
    else:
        table_out = _new(stream, (R, max_pages), torch.int32, dev) if table_out is None else table_out
        freed = _new(stream, (R, max_pages), torch.int32, dev) if freed is None else freed
        for t, n in ((table_out, "table_out"), (freed, "freed")):
            _want(t, n, torch.int32, 2, dev)
            if t.shape != shape or t.stride(1) != 1:
                raise ValueError(f"{n} must be int32 [R, max_pages] with unit column stride")
        out0, freed0 = table_out.stride(0), freed.stride(0)
    if counts is None:
        counts = _new(stream, R, torch.int32, dev)
    else:
        _want(counts, "counts", torch.int32, 1, dev)
        if counts.shape[0] != R or not counts.is_contiguous():
            raise ValueError("counts must be contiguous int32 [R]")
    wp, nbytes, workspace = _workspace(workspace, evict_pages_workspace_size(R, max_pages, ps) if workspace is None else 0,
                                       stream, dev)
    _call(dev, "qsa_evict_pages", token_weight.data_ptr(), pages, ps, page_table.data_ptr(), pts[0], max_pages,
          seq_lens.data_ptr(), keep.data_ptr(), R, keep_first, keep_last, table_out.data_ptr(), out0,
          freed.data_ptr(), freed0, counts.data_ptr(), wp, nbytes, _raw_stream(stream, dev))
    return table_out, freed, counts
