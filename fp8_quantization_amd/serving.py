"""Python binding of libbsq_serving: the paged 8-bit key/value cache with its
attention and page management, and the mixture-of-experts layer for a few
tokens over MX weights (``include/bsq_serving.h``).

Argument marshalling only, as in the package itself: names of the C ABI, sizes
of every tensor checked here because the ABI receives pointers, ``BsqError``
for a size, ``TypeError`` for a dtype, device or layout, before anything runs.
"""
import ctypes
import os
from typing import NamedTuple

import torch

from . import (MXFP4, MXFP8, SCALES_MFMA16, BsqError, _fmt, _need, _need_vec, _OFFSETS,
               _ptr, _stream_ptr, code_width, scale_shape)

KV_PAGE = 64

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbsq_serving.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run fp8_quantization_amd/build.py "
                      "(or __graft_entry__.build()) first")

_lib = ctypes.CDLL(LIB_PATH)
_i64, _i32, _p, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _p), ("v_codes", _p), ("k_scales", _p), ("v_scales", _p),
                ("num_pages", _i64), ("page_stride", _i64), ("scale_stride", _i64),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


_c = ctypes.POINTER(_Cache)
for _name, _args, _res in (
        ("kv_cache_append", [_c, _p, _i64, _p, _i64, _p, _p, _p, _i64, _i64, _i64, _i64, _i64, _p],
         _i32),
        ("kv_cache_attention", [_c, _p, _i64, _i64, _p, _p, _p, _i64, _i64, _i64, _i64, _i64, _i64,
                                _f32, _i64, _p, _i64, _p, _p, _i64, _p], _i32),
        ("kv_cache_attention_workspace", [_i64] * 8, _i64),
        ("kv_pages_copy", [_c, _p, _p, _i64, _p], _i32),
        ("kv_pages_reserve", [_p, _i64, _i64, _i64, _p, _p, _i64, _p, _p, _i64, _p, _p], _i32),
        ("kv_pages_fork", [_c, _p, _i64, _i64, _i64, _p, _p, _p, _p, _i64, _p, _p], _i32),
        ("kv_pages_free", [_p, _i64, _i64, _i64, _p, _p, _i64, _p, _i64, _p], _i32),
        ("kv_pages_compact", [_c, _p, _i64, _i64, _i64, _p, _p, _p, _i64, _p, _p, _p, _i64, _p],
         _i32),
        ("kv_pages_compact_workspace", [_i64], _i64),
        ("moe_few_tokens", [_i32, _p, _i64, _i64, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _p, _i32,
                            _p, _p, _p, _i64, _p, _i64, _p], _i32),
        ("moe_few_tokens_workspace", [_i64] * 3, _i64),
        ("bsq_serving_last_error", [], ctypes.c_char_p)):
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _res


def serving_lib() -> ctypes.CDLL:
    """The loaded ``libbsq_serving.so`` (for callers that want the raw C ABI)."""
    return _lib


def _check(status: int):
    if status != 0:
        raise BsqError(status, _lib.bsq_serving_last_error().decode())


def _size(n: int) -> int:
    if n < 0:
        raise BsqError(1, _lib.bsq_serving_last_error().decode())
    return n


class KvCache(NamedTuple):
    """A paged key/value cache: E4M3 codes and one E8M0 scale byte per (page,
    head), as uint8 tensors.  ``k_codes`` [pages, heads, D / 16, 64, 16],
    ``v_codes`` [pages, heads, D, 64] (token 16 j + 4 g + e of a page at place
    16 g + 4 j + e), ``k_scales`` and ``v_scales`` [pages, heads].  Codes are
    contiguous within a page, scales within a page's heads."""
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor


def kv_cache(num_pages: int, num_heads: int, head_dim: int, device="cuda") -> KvCache:
    """A cache of ``num_pages`` pages of 64 tokens (uninitialised: no byte is
    read before ``kv_cache_append`` has written it)."""
    if head_dim not in (64, 128, 256):
        raise BsqError(2, f"head_dim={head_dim} is not provided (64, 128 or 256)")
    if num_pages < 0 or num_heads < 1:
        raise BsqError(1, f"num_pages={num_pages} num_heads={num_heads}")

    def new(*shape):
        return torch.empty(shape, dtype=torch.uint8, device=device)
    return KvCache(new(num_pages, num_heads, head_dim // 16, KV_PAGE, 16),
                   new(num_pages, num_heads, head_dim, KV_PAGE), new(num_pages, num_heads),
                   new(num_pages, num_heads))


def _dense_after(t: torch.Tensor, dim: int) -> bool:
    """Whether the dimensions after ``dim`` lie without gaps."""
    want = 1
    for d in range(t.dim() - 1, dim, -1):
        if t.shape[d] > 1 and t.stride(d) != want:
            return False
        want *= t.shape[d]
    return True


def _cache(cache) -> _Cache:
    for name, t, dims in zip(KvCache._fields, cache, (5, 4, 2, 2)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda or \
                t.dim() != dims or not _dense_after(t, 0):
            raise TypeError(f"{name} must be a {dims}-D uint8 GPU tensor, contiguous within a page")
    k, v, ks, vs = cache
    P, H, C = k.shape[:3]
    D = 16 * C
    if tuple(k.shape) != (P, H, C, KV_PAGE, 16) or tuple(v.shape) != (P, H, D, KV_PAGE) or \
            tuple(ks.shape) != (P, H) or tuple(vs.shape) != (P, H):
        raise BsqError(1, f"shapes {tuple(k.shape)}, {tuple(v.shape)}, {tuple(ks.shape)}, "
                          f"{tuple(vs.shape)} are no cache's")

    def stride(t, least):
        return t.stride(0) if P > 1 else least
    if P > 1 and (k.stride(0) != v.stride(0) or ks.stride(0) != vs.stride(0)):
        raise TypeError("k and v must have the same stride from a page to the next")
    return _Cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), P,
                  stride(k, H * D * KV_PAGE), stride(ks, H), H, D)


def _table(block_table, kv_lens):
    """(stride, max_pages, num_seqs) of a block table and its lengths."""
    if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32 or \
            block_table.dim() != 2 or not block_table.is_cuda or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise TypeError("block_table must be a 2-D row-major int32 GPU tensor")
    S, M = block_table.shape
    _need_vec("kv_lens", kv_lens, (torch.int32,), S)
    if kv_lens.shape[0] != S:
        raise ValueError("kv_lens must have one entry per row of block_table")
    return (block_table.stride(0) if S > 1 else M), M, S


def _rows(name, x, heads, D):
    """BF16 [rows, heads, D], dense within a row: its row stride."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 3 or \
            not x.is_cuda or not _dense_after(x, 0):
        raise TypeError(f"{name} must be a 3-D bfloat16 GPU tensor, contiguous within a row")
    if heads is not None and x.shape[1] != heads or x.shape[2] != D:
        raise BsqError(1, f"{name} is {tuple(x.shape)}; its heads and width must be [{heads}, {D}]")
    return x.stride(0) if x.shape[0] > 1 else x.shape[1] * D


def _row_offsets(row_offsets, S):
    if _need_vec("row_offsets", row_offsets, _OFFSETS, S + 1).shape[0] != S + 1:
        raise ValueError("row_offsets must have one entry more than block_table has rows")
    return row_offsets


def _same_device(*tensors):
    d = tensors[0].device
    for t in tensors[1:]:
        if t is not None and t.device != d:
            raise TypeError(f"tensors on {d} and {t.device}")
    return d


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 GPU tensor")
    return workspace


def kv_cache_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, row_offsets: torch.Tensor,
                    kv_lens: torch.Tensor, block_table: torch.Tensor, max_new: int, stream=None):
    """Write new tokens: rows row_offsets[s] .. row_offsets[s + 1] of ``k`` and
    ``v`` (BF16 [rows, heads, D]) are the last tokens of sequence s, whose
    length ``kv_lens`` counts them.  ``max_new`` bounds a sequence's rows."""
    c = _cache(cache)
    stride, M, S = _table(block_table, kv_lens)
    ldk, ldv = _rows("k", k, c.num_heads, c.head_dim), _rows("v", v, c.num_heads, c.head_dim)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have the same rows")
    _row_offsets(row_offsets, S)
    dev = _same_device(cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, k, v,
                       row_offsets, kv_lens, block_table)
    _check(_lib.kv_cache_append(c, _ptr(k), ldk, _ptr(v), ldv, _ptr(row_offsets), _ptr(kv_lens),
                                _ptr(block_table), stride, M, S, k.shape[0], int(max_new),
                                _stream_ptr(stream, dev)))


def kv_cache_attention(q: torch.Tensor, cache: KvCache, row_offsets: torch.Tensor,
                       kv_lens: torch.Tensor, block_table: torch.Tensor, max_q: int, max_kv: int,
                       scale: float | None = None, window: int = 0, out=None,
                       return_lse: bool = False, lse=None, workspace=None, stream=None):
    """Causal attention of ``q`` (BF16 [rows, query heads, D]) over the cache;
    a sequence's rows are its last tokens.  ``max_q`` bounds a sequence's
    rows, ``max_kv`` its length (a hint).  ``scale`` defaults to D ** -0.5;
    ``window`` > 0 limits a row to that many tokens.  Returns out, or (out,
    lse) with ``return_lse`` (lse fp32 [rows, query heads]).  Rows that no
    sequence owns are left as they were."""
    c = _cache(cache)
    stride, M, S = _table(block_table, kv_lens)
    ldq = _rows("q", q, None, c.head_dim)
    R, Hq, D = q.shape
    _row_offsets(row_offsets, S)
    if out is None:
        out = torch.empty((R, Hq, D), dtype=torch.bfloat16, device=q.device)
    ldo = _rows("out", out, Hq, D)
    if out.shape[0] < R:
        raise BsqError(1, f"out is {tuple(out.shape)}; it must have at least {R} rows")
    if return_lse or lse is not None:
        if lse is None:
            lse = torch.empty((R, Hq), dtype=torch.float32, device=q.device)
        _need("lse", lse, torch.float32, R, Hq)
        if not lse.is_contiguous() or lse.shape[1] != Hq:
            raise TypeError("lse must be contiguous, a column per query head")
    dev = _same_device(q, cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, row_offsets,
                       kv_lens, block_table, out, lse, workspace)
    need = _size(_lib.kv_cache_attention_workspace(c.num_heads, D, Hq, S, R, int(max_q),
                                                   int(max_kv), int(window)))
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    if need:
        ws = _workspace(workspace, need, dev)
        if workspace is None:
            ws.record_stream(s)
        ws_ptr, ws_bytes = _ptr(ws), ws.numel()
    else:
        ws_ptr, ws_bytes = None, 0
    _check(_lib.kv_cache_attention(
        c, _ptr(q), ldq, Hq, _ptr(row_offsets), _ptr(kv_lens), _ptr(block_table), stride, M, S, R,
        int(max_q), int(max_kv), float(D ** -0.5 if scale is None else scale), int(window),
        _ptr(out), ldo, _ptr(lse), ws_ptr, ws_bytes, _stream_ptr(s, dev)))
    return (out, lse) if return_lse else out


def _requests(n, **vectors):
    for name, t in vectors.items():
        if _need_vec(name, t, (torch.int32,), n).numel() != n:
            raise ValueError(f"{name} must have {n} entries")


def kv_pages_copy(cache: KvCache, src: torch.Tensor, dst: torch.Tensor, stream=None):
    """Page dst[i] becomes a copy of page src[i] (int32 vectors; distinct
    destinations, none of them a source of another pair)."""
    c = _cache(cache)
    n = src.numel()
    _requests(n, src=src, dst=dst)
    dev = _same_device(cache.k_codes, src, dst)
    _check(_lib.kv_pages_copy(c, _ptr(src), _ptr(dst), n, _stream_ptr(stream, dev)))


def kv_pages_reserve(block_table: torch.Tensor, kv_lens: torch.Tensor, refcounts: torch.Tensor,
                     slots: torch.Tensor, add_tokens: torch.Tensor, status=None, stream=None):
    """Lengthen sequences slots[i] by add_tokens[i] tokens, with pages of
    refcount 0, lowest number first, requests in order.  Returns status
    (int32: 0 done, 1 no pages or table entries left, 2 no such slot)."""
    stride, M, S = _table(block_table, kv_lens)
    _need_vec("refcounts", refcounts, (torch.int32,), 0)
    n = slots.numel()
    if status is None:
        status = torch.empty(n, dtype=torch.int32, device=slots.device)
    _requests(n, slots=slots, add_tokens=add_tokens, status=status)
    dev = _same_device(block_table, kv_lens, refcounts, slots, add_tokens, status)
    _check(_lib.kv_pages_reserve(_ptr(block_table), stride, M, S, _ptr(kv_lens), _ptr(refcounts),
                                 refcounts.numel(), _ptr(slots), _ptr(add_tokens), n, _ptr(status),
                                 _stream_ptr(stream, dev)))
    return status


def _cache_refcounts(c, refcounts):
    if _need_vec("refcounts", refcounts, (torch.int32,), c.num_pages).numel() != c.num_pages:
        raise ValueError("refcounts must have one entry per page of the cache")


def kv_pages_fork(cache: KvCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                  refcounts: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
                  status=None, stream=None):
    """Slot children[i] (empty) becomes a copy of slot parents[i]: full pages
    shared, a partly filled last page copied.  Returns status as
    ``kv_pages_reserve`` does."""
    c = _cache(cache)
    stride, M, S = _table(block_table, kv_lens)
    _cache_refcounts(c, refcounts)
    n = parents.numel()
    if status is None:
        status = torch.empty(n, dtype=torch.int32, device=parents.device)
    _requests(n, parents=parents, children=children, status=status)
    dev = _same_device(cache.k_codes, block_table, kv_lens, refcounts, parents, children, status)
    _check(_lib.kv_pages_fork(c, _ptr(block_table), stride, M, S, _ptr(kv_lens), _ptr(refcounts),
                              _ptr(parents), _ptr(children), n, _ptr(status),
                              _stream_ptr(stream, dev)))
    return status


def kv_pages_free(block_table: torch.Tensor, kv_lens: torch.Tensor, refcounts: torch.Tensor,
                  slots: torch.Tensor, stream=None):
    """Sequences slots[i] give their pages back and get length 0."""
    stride, M, S = _table(block_table, kv_lens)
    _need_vec("refcounts", refcounts, (torch.int32,), 0)
    _need_vec("slots", slots, (torch.int32,), 0)
    dev = _same_device(block_table, kv_lens, refcounts, slots)
    _check(_lib.kv_pages_free(_ptr(block_table), stride, M, S, _ptr(kv_lens), _ptr(refcounts),
                              refcounts.numel(), _ptr(slots), slots.numel(),
                              _stream_ptr(stream, dev)))


def kv_pages_compact(cache: KvCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                     refcounts: torch.Tensor, table_out=None, refcounts_out=None, num_live=None,
                     workspace=None, stream=None):
    """Move the pages in use to the front of the cache.  Returns (table,
    refcounts, num_live int32 [1]); the outputs may be the inputs themselves
    (``table_out=block_table``, ``refcounts_out=refcounts``)."""
    c = _cache(cache)
    stride, M, S = _table(block_table, kv_lens)
    _cache_refcounts(c, refcounts)
    dev = refcounts.device
    if table_out is None:
        table_out = torch.empty((S, M), dtype=torch.int32, device=dev)
    if refcounts_out is None:
        refcounts_out = torch.empty_like(refcounts)
    if num_live is None:
        num_live = torch.empty(1, dtype=torch.int32, device=dev)
    out_stride, M2, S2 = _table(table_out, kv_lens)
    if (M2, S2) != (M, S):
        raise BsqError(1, f"table_out is {(S2, M2)}; it must be {(S, M)}")
    _cache_refcounts(c, refcounts_out)
    _need_vec("num_live", num_live, (torch.int32,), 1)
    _same_device(cache.k_codes, block_table, kv_lens, refcounts, table_out, refcounts_out, num_live,
                 workspace)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = _workspace(workspace, _lib.kv_pages_compact_workspace(c.num_pages), dev)
    if workspace is None:
        ws.record_stream(s)
    _check(_lib.kv_pages_compact(c, _ptr(block_table), stride, M, S, _ptr(kv_lens), _ptr(refcounts),
                                 _ptr(table_out), out_stride, _ptr(refcounts_out), _ptr(num_live),
                                 _ptr(ws), ws.numel(), _stream_ptr(s, dev)))
    return table_out, refcounts_out, num_live


def moe_few_tokens(x: torch.Tensor, fmt, w13_codes: torch.Tensor, w13_scales: torch.Tensor,
                   w2_codes: torch.Tensor, w2_scales: torch.Tensor, num_experts: int, topk: int,
                   router_logits=None, topk_ids=None, topk_weights=None, renormalize: bool = True,
                   out=None, workspace=None, stream=None):
    """A mixture-of-experts layer for at most 64 tokens: y[t] = sum over the
    token's experts of weight * W2 (silu(W1 x) * (W3 x)).  ``x`` BF16
    [tokens, hidden].  Weights: MXFP4 or MXFP8 codes with MFMA-layout scales
    (``scale_layout=SCALES_MFMA16``), w13 [experts * 2 * inter, hidden] (W1's
    rows, then W3's, per expert), w2 [experts * hidden, inter].  Routed by
    ``router_logits`` (fp32 [tokens, experts]) or by the caller's ``topk_ids``
    (int32) and ``topk_weights`` (fp32) [tokens, topk].  Returns (out,
    topk_ids, topk_weights)."""
    f = _fmt(fmt)
    if f not in (MXFP4, MXFP8):
        raise BsqError(2, f"format {fmt} is not provided (MXFP4 or MXFP8 weights)")
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 2 or \
            not x.is_cuda or (x.shape[1] > 1 and x.stride(1) != 1):
        raise TypeError("x must be a 2-D row-major bfloat16 GPU tensor")
    T, H = x.shape
    E, k = int(num_experts), int(topk)
    if E < 1 or w13_codes.shape[0] % (2 * E):
        raise BsqError(1, "w13_codes must hold num_experts * 2 * inter rows, num_experts >= 1")
    inter = w13_codes.shape[0] // (2 * E)
    if H % 128 or inter % 128:
        raise BsqError(1, f"hidden={H} and inter={inter} must be multiples of 128")
    for name, codes, scales, rows, K in (("w13_", w13_codes, w13_scales, 2 * E * inter, H),
                                         ("w2_", w2_codes, w2_scales, E * H, inter)):
        _need(name + "codes", codes, torch.uint8, rows, code_width(f, K))
        groups, width = scale_shape(f, rows, K, SCALES_MFMA16)
        _need(name + "scales", scales, torch.uint8, groups, width)
        if not codes.is_contiguous() or codes.shape[1] != code_width(f, K) or \
                not scales.is_contiguous() or scales.shape[1] != width:
            raise TypeError(f"{name}codes and {name}scales must lie without gaps")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _need("out", out, torch.bfloat16, T, H)
    if router_logits is not None:
        _need("router_logits", router_logits, torch.float32, T, E)
        if not router_logits.is_contiguous() or router_logits.shape[1] != E:
            raise TypeError("router_logits must be contiguous, a column per expert")
        if topk_ids is None:
            topk_ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
        if topk_weights is None:
            topk_weights = torch.empty((T, k), dtype=torch.float32, device=x.device)
    elif topk_ids is None or topk_weights is None:
        raise ValueError("give router_logits, or topk_ids and topk_weights")
    for name, t, dt in (("topk_ids", topk_ids, torch.int32),
                        ("topk_weights", topk_weights, torch.float32)):
        _need(name, t, dt, T, k)
        if not t.is_contiguous() or t.shape[1] != k:
            raise TypeError(f"{name} must be contiguous, topk columns")
    dev = _same_device(x, w13_codes, w13_scales, w2_codes, w2_scales, router_logits, topk_ids,
                       topk_weights, out, workspace)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    # sizes that this refuses are refused by the call below, with its message
    ws = _workspace(workspace, max(_lib.moe_few_tokens_workspace(T, inter, k), 0), dev)
    if workspace is None:
        ws.record_stream(s)
    _check(_lib.moe_few_tokens(
        f, _ptr(x), x.stride(0) if T > 1 else H, T, H, inter, E, k, _ptr(w13_codes),
        _ptr(w13_scales), _ptr(w2_codes), _ptr(w2_scales), _ptr(router_logits), int(renormalize),
        _ptr(topk_ids), _ptr(topk_weights), _ptr(out), out.stride(0) if T > 1 else H, _ptr(ws),
        ws.numel(), _stream_ptr(s, dev)))
    return out, topk_ids, topk_weights
