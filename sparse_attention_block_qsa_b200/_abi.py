"""ctypes binding of ``libqsa.so`` (the C ABI declared in include/qsa.h).

Argument marshalling only: torch tensors supply device pointers, strides and
the current stream; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the library or a GPU is missing the
calls raise.
"""
from __future__ import annotations

import ctypes as C
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
    "qsa_evict_pages_workspace_size": (_sz, [_i32, _i32]),
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


def _placed(stream, *tensors):
    """(device, stream handle) of a call on the given tensors (None skipped): they must all live on one device, and
    the call runs there, on `stream` or on that device's current stream."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}: one call needs one device")
    if stream is None:
        return dev, C.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
    return dev, _stream(stream)


def _new(stream, shape, dtype, dev):
    """Memory that belongs to the stream the call runs on (an output or a workspace made here)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _call(dev, name, *args):
    """The library call with `dev` current."""
    if dev.index == torch.cuda.current_device():
        _check(name, getattr(lib(), name)(*args))
    else:
        with torch.cuda.device(dev):
            _check(name, getattr(lib(), name)(*args))


def _workspace(workspace, need, stream, dev):
    if workspace is None:
        workspace = _new(stream, (max(need, 16),), torch.uint8, dev)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


def _cache8(k_cache, v_cache, k_scale, v_scale):
    """Check the 8-bit cache's tensors; returns (codes of K, codes of V, block_tokens)."""
    k_cache, v_cache = (c.view(torch.uint8) if isinstance(c, torch.Tensor) and c.dtype == torch.float8_e4m3fn else c
                        for c in (k_cache, v_cache))
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(k_scale, "k_scale", torch.float32, 3)
    _need(v_scale, "v_scale", torch.float32, 3)
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride() or k_cache.shape[3] != 256 \
            or k_cache.stride(3) != 1:
        raise ValueError("k_cache and v_cache must be [pages, page_size, Hkv, 256] with the same strides")
    pages, ps, Hkv, _ = k_cache.shape
    blocks = k_scale.shape[1]
    if k_scale.shape != v_scale.shape or k_scale.stride() != v_scale.stride() or k_scale.stride(2) != 1 \
            or k_scale.shape[0] != pages or k_scale.shape[2] != Hkv or blocks < 1 or ps % blocks:
        raise ValueError("k_scale and v_scale must be [pages, blocks, Hkv] with the same strides, unit head stride, "
                         "and blocks must divide page_size")
    return k_cache, v_cache, ps // blocks


def _tables(page_table, cu_seqlens_q, seq_lens):
    _need(page_table, "page_table", torch.int32, 2)
    _index_checks(cu_seqlens_q, seq_lens)
    if page_table.stride(1) != 1 or page_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("page_table needs one row per request and a unit column stride")


def _token_weight(token_weight, pages, page_size):
    _need(token_weight, "token_weight", torch.int64, 2)
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
    dt = k.dtype if isinstance(k, torch.Tensor) and k.dtype == torch.float16 else torch.bfloat16
    _need(k, "k", dt, 3)
    _need(v, "v", dt, 3)
    k_cache, v_cache, bt = _cache8(k_cache, v_cache, k_scale, v_scale)
    _tables(page_table, cu_seqlens_q, seq_lens)
    pages, ps, Hkv, _ = k_cache.shape
    if k.shape != v.shape or k.shape[1:] != (Hkv, 256) or k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("k and v must be [T, Hkv, 256] with unit feature stride")
    if token_weight is not None:
        _token_weight(token_weight, pages, ps)
    dev, st = _placed(stream, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, seq_lens,
                      token_weight)
    _call(dev, "qsa_kv_append_fp8_f16" if dt == torch.float16 else "qsa_kv_append_fp8",
          _ptr(k), k.stride(0), k.stride(1), _ptr(v), v.stride(0), v.stride(1), _ptr(k_cache), _ptr(v_cache),
          _ptr(k_scale), _ptr(v_scale), pages, ps, bt, k_cache.stride(0), k_cache.stride(1), k_cache.stride(2),
          k_scale.stride(0), k_scale.stride(1), Hkv, _ptr(page_table), page_table.stride(0), page_table.shape[1],
          _ptr(cu_seqlens_q), _ptr(seq_lens), seq_lens.shape[0], k.shape[0], _ptr(token_weight), st)


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
    dt = q.dtype if isinstance(q, torch.Tensor) and q.dtype == torch.float16 else torch.bfloat16
    _need(q, "q", dt, 3)
    k_cache, v_cache, bt = _cache8(k_cache, v_cache, k_scale, v_scale)
    _tables(page_table, cu_seqlens_q, seq_lens)
    _need(token_idx, "token_idx", torch.int32, 2)
    T, Hq, Dq = q.shape
    pages, ps, Hkv, _ = k_cache.shape
    width = token_idx.shape[1]
    if Dq != 256 or q.stride(2) != 1:
        raise ValueError("q must be [T, Hq, 256] with unit feature stride")
    if token_idx.shape[0] != T or token_idx.stride(1) != 1:
        raise ValueError("token_idx must be [T, width] with unit column stride")
    if gate is not None:
        _need(gate, "gate", torch.float32, 2)
        if gate.shape != (T, Hq) or not gate.is_contiguous():
            raise ValueError("gate must be contiguous fp32 [T, Hq]")
    if weights is not None:
        _need(weights, "weights", torch.float32, 2)
        if weights.shape != (T, width) or weights.stride(1) != 1:
            raise ValueError("weights must be fp32 [T, width] with unit column stride")
    dev, st = _placed(stream, q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, seq_lens, token_idx,
                      gate, out, lse, weights, workspace)
    if out is None:
        out = _new(stream, (T, Hq, 256), dt, dev)
    _need(out, "out", dt, 3)
    if out.shape != (T, Hq, 256) or out.stride(2) != 1 or out.stride(1) != 256:
        raise ValueError("out must be [T, Hq, 256] with contiguous heads")
    if lse is None:
        lse = _new(stream, (T, Hq), torch.float32, dev)
    _need(lse, "lse", torch.float32, 2)
    if lse.shape != (T, Hq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [T, Hq]")
    workspace, nbytes = _workspace(
        workspace, sparse_attention_fp8_workspace_size(T, Hq, Hkv, max(width, 1), weights is not None), stream, dev)
    _call(dev, "qsa_sparse_attention_fp8_f16" if dt == torch.float16 else "qsa_sparse_attention_fp8",
          _ptr(q), q.stride(0), q.stride(1), Hq, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), pages, ps,
          bt, k_cache.stride(0), k_cache.stride(1), k_cache.stride(2), k_scale.stride(0), k_scale.stride(1), Hkv,
          _ptr(page_table), page_table.stride(0), page_table.shape[1], _ptr(cu_seqlens_q), _ptr(seq_lens),
          seq_lens.shape[0], _ptr(token_idx), token_idx.stride(0), width, T, _ptr(gate), float(scale), _ptr(out),
          out.stride(0), _ptr(lse), _ptr(weights), weights.stride(0) if weights is not None else 0, _ptr(workspace),
          nbytes, st)
    return out, lse


def accumulate_weights(weights: torch.Tensor, token_idx: torch.Tensor, page_table: torch.Tensor,
                       cu_seqlens_q: torch.Tensor, seq_lens: torch.Tensor, token_weight: torch.Tensor,
                       stream=None) -> torch.Tensor:
    """Add attention weights (fp32 [T, width], one per entry of token_idx int32 [T, width]) up per cached token, in
    place: token_weight int64 [pages, page_size] in units of 2^-32.  Returns token_weight."""
    _need(weights, "weights", torch.float32, 2)
    _need(token_idx, "token_idx", torch.int32, 2)
    _need(token_weight, "token_weight", torch.int64, 2)
    _tables(page_table, cu_seqlens_q, seq_lens)
    pages, ps = token_weight.shape
    _token_weight(token_weight, pages, ps)
    T, width = token_idx.shape
    if weights.shape != (T, width) or weights.stride(1) != 1 or token_idx.stride(1) != 1:
        raise ValueError("weights and token_idx must be [T, width] with unit column strides")
    dev, st = _placed(stream, weights, token_idx, page_table, cu_seqlens_q, seq_lens, token_weight)
    _call(dev, "qsa_accumulate_weights", _ptr(weights), weights.stride(0), _ptr(token_idx), token_idx.stride(0), width,
          T, _ptr(page_table), page_table.stride(0), page_table.shape[1], _ptr(cu_seqlens_q), _ptr(seq_lens),
          seq_lens.shape[0], _ptr(token_weight), pages, ps, st)
    return token_weight


def evict_pages_workspace_size(R: int, max_pages: int) -> int:
    return int(lib().qsa_evict_pages_workspace_size(R, max_pages))


def evict_pages(token_weight: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, keep: torch.Tensor,
                keep_first: int = 0, keep_last: int = 1, table_out: torch.Tensor | None = None,
                freed: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """Drop the pages of least accumulated weight (token_weight int64 [pages, page_size]) until request r has
    keep[r] (int32 [R]) live pages; its first keep_first and last keep_last logical pages stay.  Returns (table_out
    int32 [R, max_pages] with -1 for dropped pages, freed int32 [R, max_pages]: the dropped pages in order, then -1,
    counts int32 [R]).  table_out may be page_table."""
    _need(token_weight, "token_weight", torch.int64, 2)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(keep, "keep", torch.int32, 1)
    pages, ps = token_weight.shape
    _token_weight(token_weight, pages, ps)
    R, max_pages = page_table.shape
    if seq_lens.shape[0] != R or keep.shape[0] != R or not seq_lens.is_contiguous() or not keep.is_contiguous() \
            or page_table.stride(1) != 1:
        raise ValueError("page_table needs one row per request and a unit column stride, seq_lens and keep one "
                         "contiguous entry per request")
    dev, st = _placed(stream, token_weight, page_table, seq_lens, keep, table_out, freed, counts, workspace)
    table_out = _new(stream, (R, max_pages), torch.int32, dev) if table_out is None else table_out
    freed = _new(stream, (R, max_pages), torch.int32, dev) if freed is None else freed
    counts = _new(stream, (R,), torch.int32, dev) if counts is None else counts
    for t, n in ((table_out, "table_out"), (freed, "freed")):
        _need(t, n, torch.int32, 2)
        if t.shape != (R, max_pages) or t.stride(1) != 1:
            raise ValueError(f"{n} must be int32 [R, max_pages] with unit column stride")
    _need(counts, "counts", torch.int32, 1)
    if counts.shape[0] != R or not counts.is_contiguous():
        raise ValueError("counts must be contiguous int32 [R]")
    workspace, nbytes = _workspace(workspace, evict_pages_workspace_size(R, max_pages), stream, dev)
    _call(dev, "qsa_evict_pages", _ptr(token_weight), pages, ps, _ptr(page_table), page_table.stride(0), max_pages,
          _ptr(seq_lens), _ptr(keep), R, int(keep_first), int(keep_last), _ptr(table_out), table_out.stride(0),
          _ptr(freed), freed.stride(0), _ptr(counts), _ptr(workspace), nbytes, st)
    return table_out, freed, counts
