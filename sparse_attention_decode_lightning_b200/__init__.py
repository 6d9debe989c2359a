"""Thin Python binding of libdsa (DSA decode on B200, sm_100a).

Argument marshalling only: every function below forwards torch tensors'
device pointers to the C ABI declared in include/dsa.h, under the same name,
and raises DSAError on a non-zero status.  No step of the computation runs in
Python, and there is no fallback: if libdsa.so is missing, loading fails.
"""
import ctypes
import operator
import os
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

PAGE_SIZE = 64
TIER_PAGE = 16       # tokens per slot of the two-tier (HiSparse) cache
HEADS = 128          # MLA heads, DeepSeek-V3.2
HEADS_GLM = 64       # MLA heads, GLM-5.2
DIM = 576
DIM_V = 512
IDX_HEADS = 64       # indexer heads, DeepSeek-V3.2
IDX_HEADS_GLM = 32   # indexer heads, GLM-5.2
IDX_DIM = 128
MAX_TOPK = 2048
MAX_Q_PER_SEQ = 8

STATUS = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_CUDA",
          4: "DSA_ERR_DEVICE_BOUNDS", 5: "DSA_ERR_TIMEOUT", 6: "DSA_ERR_WORKSPACE"}

# name -> (restype, argtypes) of every exported entry point
_P, _I, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_PP = ctypes.POINTER(ctypes.c_void_p)
SIGNATURES = {
    "dsa_status_string": (ctypes.c_char_p, [_I]),
    "dsa_version": (_I, []),
    "dsa_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "dsa_choose_splits": (_I, [_I, _I, _I]),
    "dsa_mla_group_plan": (_I, [_I, _I, _P, _P, _P]),
    "dsa_indexer_scores": (_I, [_P, _P, _P, _I64, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P, _SZ,
                                _P]),
    "dsa_topk_select": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "dsa_indexer_topk": (_I, [_P, _P, _P, _I64, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _SZ,
                              _P]),
    "dsa_indexer_topk_fused": (_I, [_P, _P, _P, _I64, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P,
                                    _P, _SZ, _P]),
    "dsa_sparse_mla_decode": (_I, [_P, _P, _I, _I, _P, _I, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P,
                                   _P, _P, _SZ, _P]),
    "dsa_sparse_mla_decode_noalloc": (_I, [_P, _P, _I, _I, _P, _I, _P, _P, _P, _I, _I, _I, _I, _F,
                                           _I, _P, _P, _P]),
    "dsa_sparse_mla_decode_window": (_I, [_P, _P, _I, _I, _P, _I, _P, _I, _P, _P, _P, _P, _I, _I,
                                          _I, _I, _I, _F, _I, _P, _P, _P, _SZ, _P]),
    "dsa_sparse_mla_decode_fp8": (_I, [_P, _P, _F, _I, _I, _P, _I, _P, _P, _P, _I, _I, _I, _I, _F,
                                       _I, _P, _P, _P, _SZ, _P]),
    "dsa_latent_append": (_I, [_P, _I64, _P, _I64, _P, _I, _P, _I, _P, _P, _I, _I, _P, _P, _I, _I,
                               _I, _P, _SZ, _P]),
    "dsa_attend_workspace_bytes": (_SZ, [_I]),
    "dsa_mla_decode_sinks": (_I, [_P, _P, _P, _I, _I, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _F,
                                  _P, _P, _P, _SZ, _P]),
    "dsa_sparse_mla_decode_fp8_block": (_I, [_P, _P, _P, _I, _I, _I, _P, _I, _P, _P, _P, _I, _I, _I,
                                             _I, _F, _P, _P, _P, _SZ, _P]),
    "dsa_lse_combine": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "dsa_decode_step": (_I, [_I, _I, _I, _PP, _PP, _PP, _I64, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                             _PP, _PP, _I, _I, _PP, _I, _F, _I, _PP, _PP, _P, _P, _SZ, _P]),
    "dsa_tier_state_bytes": (_SZ, [_I, _I, _I]),
    "dsa_tier_init": (_I, [_P, _SZ, _I, _I, _I]),
    "dsa_tier_plan": (_I, [_P, _P, _I, _I, _P, _P, _P, _I, _P, _P]),
    "dsa_tier_fetch": (_I, [_P, _I64, _P, _I64, _P, _I, _P, _P, _P]),
    "dsa_tier_dev_state_bytes": (_SZ, [_I, _I, _I]),
    "dsa_tier_dev_init": (_I, [_P, _SZ, _I, _I, _I, _P, _P]),
    "dsa_tier_swap_in": (_I, [_P, _SZ, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P]),
    "dsa_tier_dev_stats": (_I, [_P, _P, _P]),
    "dsa_tier_dev_copies": (_P, [_P, _I, _I, _I]),
    "dsa_check_error": (_I, [_P, _P]),
    "dsa_noalloc_check_error": (_I, [_P]),
    "dsa_selftest_bounded_wait": (_I, [_I, _P, _SZ, _P]),
}

_lib = None


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


def lib() -> ctypes.CDLL:
    """Load libdsa.so (built in-tree by build.py); fails loudly if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_attention_decode_lightning_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libdsa takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libdsa takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _host_ptr(t: torch.Tensor):
    if t.is_cuda:
        raise ValueError("this argument is host memory")
    if not t.is_contiguous():
        raise ValueError("libdsa takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(status: int, where: str):
    if status != 0:
        raise DSAError(status, where)


def _ptr_array(ts: Sequence[Optional[torch.Tensor]]):
    arr = (ctypes.c_void_p * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = None if t is None else _ptr(t).value
    return arr


def dsa_version() -> int:
    return lib().dsa_version()


def dsa_status_string(s: int) -> str:
    return lib().dsa_status_string(s).decode()


def dsa_choose_splits(Q: int, topk: int, num_splits: int = 0) -> int:
    return lib().dsa_choose_splits(Q, topk, num_splits)


def dsa_mla_group_plan(units: int, topk: int):
    """(head_units, tail_units, tail_splits) of an IndexShare group's grouped
    attention, or None for invalid sizes."""
    h, t, ts = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    if not lib().dsa_mla_group_plan(units, topk, ctypes.byref(h), ctypes.byref(t), ctypes.byref(ts)):
        return None
    return h.value, t.value, ts.value


def dsa_workspace_bytes(Q: int, max_len: int, topk: int, num_splits: int = 0) -> int:
    return lib().dsa_workspace_bytes(Q, max_len, topk, num_splits)


def workspace(Q: int, max_len: int, topk: int, num_splits: int = 0, device="cuda") -> torch.Tensor:
    """A zeroed device workspace of dsa_workspace_bytes(...) bytes."""
    n = dsa_workspace_bytes(Q, max_len, topk, num_splits)
    if n == 0:
        raise DSAError(1, "dsa_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def dsa_indexer_scores(q_idx, w, k_idx, seq_offsets, q_offsets, q_vis, B, max_len, scores, ws,
                       first_only=False, stream=None):
    _check(lib().dsa_indexer_scores(
        _ptr(q_idx), _ptr(w), _ptr(k_idx), k_idx.shape[0], _ptr(seq_offsets), _ptr(q_offsets),
        _ptr(q_vis), B, q_idx.shape[0], q_idx.shape[1], max_len, int(first_only), _ptr(scores),
        scores.shape[1], _ptr(ws), ws.numel(), _stream(stream)), "dsa_indexer_scores")


def dsa_topk_select(scores, q_offsets, q_vis, B, max_len, topk, out_idx, ws, out_scores=None,
                    first_only=False, stream=None):
    _check(lib().dsa_topk_select(
        _ptr(scores), scores.shape[1], _ptr(q_offsets), _ptr(q_vis), B, scores.shape[0], max_len,
        topk, int(first_only), _ptr(out_idx), _ptr(out_scores), _ptr(ws), ws.numel(),
        _stream(stream)), "dsa_topk_select")


def dsa_indexer_topk(q_idx, w, k_idx, seq_offsets, q_offsets, q_vis, B, max_len, topk, out_idx,
                     ws, out_scores=None, first_only=False, stream=None):
    _check(lib().dsa_indexer_topk(
        _ptr(q_idx), _ptr(w), _ptr(k_idx), k_idx.shape[0], _ptr(seq_offsets), _ptr(q_offsets),
        _ptr(q_vis), B, q_idx.shape[0], q_idx.shape[1], max_len, topk, int(first_only),
        _ptr(out_idx), _ptr(out_scores), _ptr(ws), ws.numel(), _stream(stream)), "dsa_indexer_topk")


def dsa_indexer_topk_fused(q_idx, w, k_idx, seq_offsets, q_offsets, q_vis, B, max_len, topk,
                           out_idx, ws, out_scores=None, first_only=False, stream=None):
    _check(lib().dsa_indexer_topk_fused(
        _ptr(q_idx), _ptr(w), _ptr(k_idx), k_idx.shape[0], _ptr(seq_offsets), _ptr(q_offsets),
        _ptr(q_vis), B, q_idx.shape[0], q_idx.shape[1], max_len, topk, int(first_only),
        _ptr(out_idx), _ptr(out_scores), _ptr(ws), ws.numel(), _stream(stream)),
        "dsa_indexer_topk_fused")


def dsa_sparse_mla_decode(q, kv_pool, page_table, q_offsets, q_vis, idx, B, scale, out, lse, ws,
                          num_splits=0, stream=None):
    _check(lib().dsa_sparse_mla_decode(
        _ptr(q), _ptr(kv_pool), kv_pool.shape[0], kv_pool.shape[1], _ptr(page_table),
        page_table.shape[1],
        _ptr(q_offsets), _ptr(q_vis), _ptr(idx), B, q.shape[0], q.shape[1], idx.shape[1],
        float(scale), num_splits, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
        "dsa_sparse_mla_decode")


def dsa_sparse_mla_decode_noalloc(q, kv_pool, page_table, q_offsets, q_vis, idx, B, scale, out,
                                  lse, num_splits=0, stream=None):
    """dsa_sparse_mla_decode without a workspace (split-K partials in the
    library's own fixed device array; see include/dsa.h)."""
    _check(lib().dsa_sparse_mla_decode_noalloc(
        _ptr(q), _ptr(kv_pool), kv_pool.shape[0], kv_pool.shape[1], _ptr(page_table),
        page_table.shape[1],
        _ptr(q_offsets), _ptr(q_vis), _ptr(idx), B, q.shape[0], q.shape[1], idx.shape[1],
        float(scale), num_splits, _ptr(out), _ptr(lse), _stream(stream)),
        "dsa_sparse_mla_decode_noalloc")


def dsa_sparse_mla_decode_window(q, kv_pool, page_table, win_page_table, q_offsets, q_vis,
                                 win_vis, idx, B, window, scale, out, lse, ws, num_splits=0,
                                 stream=None):
    """Sparse MLA over the selected compressed entries plus a sliding window of
    raw tokens (DeepSeek-V4 CSA); see include/dsa.h."""
    _check(lib().dsa_sparse_mla_decode_window(
        _ptr(q), _ptr(kv_pool), kv_pool.shape[0], kv_pool.shape[1], _ptr(page_table),
        page_table.shape[1], _ptr(win_page_table), win_page_table.shape[1], _ptr(q_offsets),
        _ptr(q_vis), _ptr(win_vis), _ptr(idx), B, q.shape[0], q.shape[1], idx.shape[1], window,
        float(scale), num_splits, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
        "dsa_sparse_mla_decode_window")


def dsa_sparse_mla_decode_fp8(q, kv_pool, kv_scale, page_table, q_offsets, q_vis, idx, B, scale,
                              out, lse, ws, num_splits=0, stream=None):
    """Sparse MLA over an e4m3 latent cache (uint8 [pages,page_size,576]) with one
    per-tensor scale; see include/dsa.h."""
    _check(lib().dsa_sparse_mla_decode_fp8(
        _ptr(q), _ptr(kv_pool), float(kv_scale), kv_pool.shape[0], kv_pool.shape[1],
        _ptr(page_table), page_table.shape[1], _ptr(q_offsets), _ptr(q_vis), _ptr(idx), B,
        q.shape[0], q.shape[1], idx.shape[1], float(scale), num_splits, _ptr(out), _ptr(lse),
        _ptr(ws), ws.numel(), _stream(stream)), "dsa_sparse_mla_decode_fp8")


# The calls below cost a decode step a few microseconds of host time each, so
# they check their arguments once, with few operations on each tensor.
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
_E4M3 = (torch.uint8, torch.float8_e4m3fn)


def _device_of(t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("libdsa takes device tensors")
    if dev != torch._C._cuda_getDevice():            # a device tensor exists, so CUDA is initialised
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device")
    return dev


def _bad(name: str, t: torch.Tensor, dtype, shape, dev: int):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the others are on cuda:{dev}")
    raise ValueError(f"{name}: libdsa takes contiguous tensors")


def _at(name: str, t: torch.Tensor, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on device `dev`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _bad(name, t, dtype, shape, dev)


def _rows_at(name: str, t: torch.Tensor, width: int, dev: int) -> int:
    """Address of a bf16 [T, width] tensor whose rows may be apart."""
    if t.dtype is not _BF16 or t.dim() != 2 or t.shape[1] != width or t.stride(1) != 1:
        raise ValueError(f"{name}: [T, {width}] {_BF16} with dense rows")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the others are on cuda:{dev}")
    return t.data_ptr()


def _ws_at(ws: torch.Tensor, dev: int):
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: a contiguous tensor on cuda:{dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _tokens(name: str, n) -> int:
    """A count of tokens as the C call's int, which keeps the lower 32 bits of a larger one: no context is
    longer than its largest value."""
    n = operator.index(n)
    if n < 0:
        raise ValueError(f"{name}: expected 0 or more, got {n}")
    return n if n < 0x7FFFFFFF else 0x7FFFFFFF


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _cache(kv_pool, kv_scales, page_table, q_offsets, q_vis, rows: int, B: int, dev: int):
    """Checks the latent cache and the bookkeeping of a call; returns the C call's
    (pool, scales, num_pages, page_size, tokens of a scale), (table, max_pages), offsets, vis."""
    if kv_pool.dim() != 3:
        raise ValueError("kv_pool: [num_pages, page_size, 576]")
    pages, page = kv_pool.shape[0], kv_pool.shape[1]
    shape = (pages, page, DIM)
    if kv_scales is None:
        pool, scales, block = _at("kv_pool", kv_pool, _BF16, shape, dev), None, 1
    else:
        if kv_pool.dtype not in _E4M3:
            raise ValueError(f"kv_pool: expected {_E4M3}, got {kv_pool.dtype}")
        pool = _at("kv_pool", kv_pool, kv_pool.dtype, shape, dev)
        n = kv_scales.shape[1] if kv_scales.dim() == 2 else 0
        if n == 0 or page % n:
            raise ValueError("kv_scales: [num_pages, page_size / block]")
        scales, block = _at("kv_scales", kv_scales, _F32, (pages, n), dev), page // n
    if page_table.dim() != 2:
        raise ValueError("page_table: [B, max_pages]")
    max_pages = page_table.shape[1]
    return ((pool, scales, pages, page, block), (_at("page_table", page_table, _I32, (B, max_pages), dev), max_pages),
            _at("q_offsets", q_offsets, _I32, (B + 1,), dev), _at("q_vis", q_vis, _I32, (rows,), dev))


def dsa_latent_append(kv, k_pe, inv_freq, kv_pool, page_table, q_offsets, q_vis, B, ws,
                      kv_scales=None, interleaved=False, stream=None):
    """Appends tokens to the latent cache, the RoPE part rotated on the way: row t
    is the token at position q_vis[t] - 1 of its sequence.  kv [T,512] and k_pe
    [T,64] bf16 may be slices of one projection's output.  kv_scales (fp32
    [num_pages, page_size / block]) makes it an e4m3 cache with a scale for each
    block of tokens; see include/dsa.h."""
    dev = _device_of(kv)
    p_kv, p_pe = _rows_at("kv", kv, DIM_V, dev), _rows_at("k_pe", k_pe, DIM - DIM_V, dev)
    T = kv.shape[0]
    if k_pe.shape[0] != T:
        raise ValueError(f"k_pe: expected {T} rows, got {k_pe.shape[0]}")
    freq = _at("inv_freq", inv_freq, _F32, ((DIM - DIM_V) // 2,), dev)
    (pool, scales, pages, page, block), (table, max_pages), off, vis = _cache(kv_pool, kv_scales, page_table, q_offsets,
                                                                              q_vis, T, B, dev)
    # a single row's stride says nothing about the rows after it
    ld_kv, ld_pe = (kv.stride(0), k_pe.stride(0)) if T > 1 else (DIM_V, DIM - DIM_V)
    p_ws, n_ws = _ws_at(ws, dev)
    status = (_lib or lib()).dsa_latent_append(p_kv, ld_kv, p_pe, ld_pe, freq, 1 if interleaved else 0, table, max_pages, off,
                                               vis, B, T, pool, scales, pages, page, block, p_ws, n_ws,
                                               _raw_stream(stream, dev))
    if status:
        raise DSAError(status, "dsa_latent_append")


def dsa_attend_workspace_bytes(heads: int) -> int:
    return lib().dsa_attend_workspace_bytes(heads)


def attend_workspace(heads: int = HEADS, device="cuda") -> torch.Tensor:
    """A zeroed device workspace for dsa_mla_decode_sinks and
    dsa_sparse_mla_decode_fp8_block (one for 128 heads also serves 64)."""
    n = dsa_attend_workspace_bytes(heads)
    if n == 0:
        raise DSAError(2, "dsa_attend_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def dsa_mla_decode_sinks(q, kv_pool, page_table, q_offsets, q_vis, B, sinks, window, scale, out,
                         lse, ws, kv_scales=None, stream=None):
    """MLA decode over the first `sinks` and the last `window` visible tokens, of a
    bf16 cache or (kv_scales) a block-scaled e4m3 one; a window of any size at least
    the context is dense attention.  out bf16 [Q,heads,512], lse fp32 [Q,heads]; see
    include/dsa.h."""
    dev = _device_of(q)
    if q.dim() != 3:
        raise ValueError("q: [Q, heads, 576]")
    Q, H = q.shape[0], q.shape[1]
    (pool, scales, pages, page, block), (table, max_pages), off, vis = _cache(kv_pool, kv_scales, page_table, q_offsets,
                                                                              q_vis, Q, B, dev)
    p_ws, n_ws = _ws_at(ws, dev)
    status = (_lib or lib()).dsa_mla_decode_sinks(
        _at("q", q, _BF16, (Q, H, DIM), dev), pool, scales, pages, page, block, table, max_pages, off, vis, B, Q, H,
        _tokens("sinks", sinks), _tokens("window", window), scale, _at("out", out, _BF16, (Q, H, DIM_V), dev), _at("lse", lse, _F32, (Q, H), dev), p_ws, n_ws,
        _raw_stream(stream, dev))
    if status:
        raise DSAError(status, "dsa_mla_decode_sinks")


def dsa_sparse_mla_decode_fp8_block(q, kv_pool, kv_scales, page_table, q_offsets, q_vis, idx, B,
                                    scale, out, lse, ws, stream=None):
    """Sparse MLA over the selected tokens of a block-scaled e4m3 cache; out bf16
    [Q,heads,512], lse fp32 [Q,heads]; see include/dsa.h."""
    dev = _device_of(q)
    if q.dim() != 3 or idx.dim() != 2 or kv_scales is None:
        raise ValueError("q: [Q, heads, 576], idx: [Q, topk], kv_scales: [num_pages, page_size / block]")
    Q, H, topk = q.shape[0], q.shape[1], idx.shape[1]
    (pool, scales, pages, page, block), (table, max_pages), off, vis = _cache(kv_pool, kv_scales, page_table, q_offsets,
                                                                              q_vis, Q, B, dev)
    p_ws, n_ws = _ws_at(ws, dev)
    status = (_lib or lib()).dsa_sparse_mla_decode_fp8_block(
        _at("q", q, _BF16, (Q, H, DIM), dev), pool, scales, pages, page, block, table, max_pages, off, vis,
        _at("idx", idx, _I32, (Q, topk), dev), B, Q, H, topk, scale, _at("out", out, _BF16, (Q, H, DIM_V), dev),
        _at("lse", lse, _F32, (Q, H), dev), p_ws, n_ws, _raw_stream(stream, dev))
    if status:
        raise DSAError(status, "dsa_sparse_mla_decode_fp8_block")


def dsa_lse_combine(o_parts, lse_parts, out, lse, stream=None):
    Q, S, H = lse_parts.shape[0], lse_parts.shape[1], lse_parts.shape[2]
    _check(lib().dsa_lse_combine(_ptr(o_parts), _ptr(lse_parts), Q, S, H, _ptr(out), _ptr(lse),
                                 _stream(stream)), "dsa_lse_combine")


def dsa_decode_step(q_idx_layers, w_layers, k_idx_layers, seq_offsets, q_offsets, q_vis, B,
                    max_len, topk, q_layers, pool_layers, page_table_layers, scale, out_layers,
                    lse_layers, idx_out, ws, index_share=1, mtp_index_share=False, num_splits=0,
                    stream=None):
    """Per-layer lists; entries of the indexer lists for non-indexer layers may be None."""
    n = len(q_layers)
    lead = next(t for t in k_idx_layers if t is not None)
    lead_q = next(t for t in q_idx_layers if t is not None)
    _check(lib().dsa_decode_step(
        n, index_share, int(mtp_index_share), _ptr_array(q_idx_layers), _ptr_array(w_layers),
        _ptr_array(k_idx_layers), lead.shape[0], _ptr(seq_offsets), _ptr(q_offsets), _ptr(q_vis),
        B, q_layers[0].shape[0], q_layers[0].shape[1], lead_q.shape[1], max_len, topk,
        _ptr_array(q_layers), _ptr_array(pool_layers),
        pool_layers[0].shape[0], pool_layers[0].shape[1], _ptr_array(page_table_layers),
        page_table_layers[0].shape[1],
        float(scale), num_splits, _ptr_array(out_layers), _ptr_array(lse_layers), _ptr(idx_out),
        _ptr(ws), ws.numel(), _stream(stream)), "dsa_decode_step")


def dsa_tier_state_bytes(B: int, dev_slots: int, max_pages: int) -> int:
    return lib().dsa_tier_state_bytes(B, dev_slots, max_pages)


def tier_state(B: int, dev_slots: int, max_pages: int) -> torch.Tensor:
    """Host memory for a two-tier cache's state, initialised (every slot empty)."""
    n = dsa_tier_state_bytes(B, dev_slots, max_pages)
    if n == 0:
        raise DSAError(1, "dsa_tier_state_bytes")
    st = torch.empty((n + 7) // 8, dtype=torch.int64)      # 8-byte aligned host bytes
    dsa_tier_init(st, B, dev_slots, max_pages)
    return st


def dsa_tier_init(state: torch.Tensor, B: int, dev_slots: int, max_pages: int):
    _check(lib().dsa_tier_init(_host_ptr(state), state.numel() * state.element_size(), B,
                               dev_slots, max_pages), "dsa_tier_init")


def dsa_tier_plan(state, idx, q_offsets, copies, page_table=None):
    """Host tensors: idx int32 [Q,topk], q_offsets int32 [B+1], copies int32
    [cap,3] (out), page_table None or int32 [B,max_pages] (out).  Returns
    (n_copies, (hits, misses, evictions))."""
    n = ctypes.c_int(0)
    stats = (ctypes.c_int64 * 3)()
    _check(lib().dsa_tier_plan(_host_ptr(state), _host_ptr(idx), idx.shape[0], idx.shape[1],
                               _host_ptr(q_offsets),
                               None if page_table is None else _host_ptr(page_table),
                               _host_ptr(copies), copies.shape[0], ctypes.byref(n), stats),
           "dsa_tier_plan")
    return n.value, (stats[0], stats[1], stats[2])


def dsa_tier_fetch(host_cache, dev_pool, copies, n, ws, page_table=None, stream=None):
    """host_cache: pinned host tensor [host_pages,16,576] bf16; dev_pool: device
    tensor [dev_pages,16,576] bf16; copies: device int32 [>=n,3]; page_table:
    None or the device int32 [B,max_pages] table to patch."""
    if not host_cache.is_pinned():
        raise ValueError("host_cache must be pinned host memory")
    _check(lib().dsa_tier_fetch(_host_ptr(host_cache), host_cache.shape[0], _ptr(dev_pool),
                                dev_pool.shape[0], _ptr(copies), n, _ptr(page_table), _ptr(ws),
                                _stream(stream)), "dsa_tier_fetch")


def tier_dev_state(B: int, dev_slots: int, max_pages: int, page_table, stream=None) -> torch.Tensor:
    """Device memory for the on-device planner's state, initialised; page_table
    (device int32 [B,max_pages]) is set to all -1."""
    n = lib().dsa_tier_dev_state_bytes(B, dev_slots, max_pages)
    if n == 0:
        raise DSAError(2, "dsa_tier_dev_state_bytes")
    st = torch.empty(n, dtype=torch.uint8, device=page_table.device)
    _check(lib().dsa_tier_dev_init(_ptr(st), n, B, dev_slots, max_pages, _ptr(page_table),
                                   _stream(stream)), "dsa_tier_dev_init")
    return st


def dsa_tier_swap_in(dev_state, B, dev_slots, max_pages, idx, q_offsets, page_table, host_cache,
                     dev_pool, ws, stream=None):
    """Plan on the device and fetch: idx device int32 [Q,topk], q_offsets device
    int32 [B+1], page_table device int32 [B,max_pages] (updated), host_cache
    pinned host bf16 [B*max_pages,16,576], dev_pool device bf16 [B*dev_slots,16,576]."""
    if not host_cache.is_pinned():
        raise ValueError("host_cache must be pinned host memory")
    _check(lib().dsa_tier_swap_in(_ptr(dev_state), dev_state.numel(), B, dev_slots, max_pages,
                                  _ptr(idx), idx.shape[0], idx.shape[1], _ptr(q_offsets),
                                  _ptr(page_table), _host_ptr(host_cache), _ptr(dev_pool), _ptr(ws),
                                  _stream(stream)), "dsa_tier_swap_in")


def dsa_tier_dev_stats(dev_state, stream=None):
    """(n_copies, hits, misses, evictions) of the last device step, and the step count."""
    out = (ctypes.c_int64 * 5)()
    _check(lib().dsa_tier_dev_stats(_ptr(dev_state), out, _stream(stream)), "dsa_tier_dev_stats")
    return tuple(out[:4]), out[4]


def dsa_tier_dev_copies(dev_state, B, dev_slots, max_pages, n):
    """The device planner's copy list (int32 [n,3]) as a tensor view of dev_state."""
    p = lib().dsa_tier_dev_copies(_ptr(dev_state), B, dev_slots, max_pages)
    off = p - dev_state.data_ptr()
    return dev_state[off:off + 12 * n].view(torch.int32).view(n, 3)


def dsa_check_error(ws, stream=None):
    _check(lib().dsa_check_error(_ptr(ws), _stream(stream)), "dsa_check_error")


def dsa_selftest_bounded_wait(limit_us, ws, stream=None):
    """Makes the library's bounded device-side waits run out (see include/dsa.h)."""
    _check(lib().dsa_selftest_bounded_wait(int(limit_us), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_selftest_bounded_wait")


def dsa_noalloc_check_error(stream=None):
    """Reads and clears dsa_sparse_mla_decode_noalloc's error word (synchronises)."""
    _check(lib().dsa_noalloc_check_error(_stream(stream)), "dsa_noalloc_check_error")
