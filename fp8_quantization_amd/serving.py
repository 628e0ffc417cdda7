"""Python binding of libbsq_serving: the paged 8-bit key/value cache with its
attention and page management, the mixture-of-experts layer for a few tokens
over MX weights (``include/bsq_serving.h``), and the operators around them in a
decoder's step (``include/bsq_decoder.h``).

Argument marshalling only, as in the package itself.  A decode step calls
these for a few microseconds of GPU work each, so the checks and the launch
are in a native module (``csrc/bsq_serving_py.cpp``): through ctypes, checking
eight to ten tensors took 18 to 30 us a call.  A size that does not fit raises
``BsqError``, a wrong dtype, device or layout ``TypeError``, before anything
runs.  Kernels run on ``stream``, or on torch's current stream.  With another
stream than the current one, as in torch: the inputs must be ready on it (and
stay until it has read them), the results are ready once the current stream
waits for it; outputs and workspaces that a call allocates are that stream's.
"""
import ctypes
import os
from typing import NamedTuple

import torch

from . import BsqError, _fmt

KV_PAGE = 64

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsq_serving.so")

for _path in (LIB_PATH, os.path.join(_HERE, "_serving.so")):
    if not os.path.exists(_path):
        raise ImportError(f"{_path} is not built; run fp8_quantization_amd/build.py "
                          "(or __graft_entry__.build()) first")

_lib = ctypes.CDLL(LIB_PATH)
_i64, _i32, _p, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
for _name, _res, *_args in (
        ("kv_cache_append", _i32, _p, _p, _i64, _p, _i64, _p, _p, _p, *[_i64] * 5, _p),
        ("kv_cache_attention", _i32, _p, _p, _i64, _i64, _p, _p, _p, *[_i64] * 6, _f32, _i64, _p,
         _i64, _p, _p, _i64, _p),
        ("kv_cache_attention_workspace", _i64, *[_i64] * 8),
        ("kv_pages_copy", _i32, _p, _p, _p, _i64, _p),
        ("kv_pages_reserve", _i32, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _p, _i64, _p, _p),
        ("kv_pages_fork", _i32, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _i64, _p, _p),
        ("kv_pages_free", _i32, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _i64, _p),
        ("kv_pages_compact", _i32, _p, _p, _i64, _i64, _i64, _p, _p, _p, _i64, _p, _p, _p, _i64,
         _p),
        ("kv_pages_compact_workspace", _i64, _i64),
        ("moe_few_tokens", _i32, _i32, _p, *[_i64] * 6, _p, _p, _p, _p, _p, _i32, _p, _p, _p, _i64,
         _p, _i64, _p),
        ("moe_few_tokens_workspace", _i64, *[_i64] * 4),
        ("kv_cache_attention_masked", _i32, _p, _p, _i64, _i64, _p, _p, _p, *[_i64] * 6, _f32, _i64,
         _i64, _p, _i64, _p, _i64, _p, _p, _i64, _p),
        ("kv_cache_attention_masked_workspace", _i64, *[_i64] * 10),
        ("qk_norm_rope", _i32, _i32, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _i64, _p, _p,
         _f32, _p, _p, _i64, _i32, _p, _i64, _p, _i64, _p, _i64, _p),
        ("moe_route", _i32, _i32, _p, *[_i64] * 4, _i32, _p, _i64, _i64, _i32, _i32, _f32, _p, _p, _p),
        ("moe_group_rows", _i32, _p, *[_i64] * 4, _p, _p, _p, _p, _p, _i64, _p),
        ("moe_group_rows_workspace", _i64, *[_i64] * 3),
        ("token_logprobs", _i32, _i32, _p, _i64, _i64, _i64, _p, _i64, _i64, _p, _p, _p, _p, _p, _i64,
         _p),
        ("token_logprobs_workspace", _i64, *[_i64] * 3),
        ("bsq_serving_last_error", ctypes.c_char_p)):
    getattr(_lib, _name).restype, getattr(_lib, _name).argtypes = _res, _args

from . import _serving  # noqa: E402  (built beside LIB_PATH, which it links)

_serving.init(BsqError)


def serving_lib() -> ctypes.CDLL:
    """The loaded ``libbsq_serving.so`` (for callers that want the raw C ABI)."""
    return _lib


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
    used before ``kv_cache_append`` has written it)."""
    if head_dim not in (64, 128, 256):
        raise BsqError(2, f"head_dim={head_dim} is not provided (64, 128 or 256)")
    if num_pages < 0 or num_heads < 1:
        raise BsqError(1, f"num_pages={num_pages} must be >= 0 and num_heads={num_heads} >= 1")

    def new(*shape):
        return torch.empty(shape, dtype=torch.uint8, device=device)
    return KvCache(new(num_pages, num_heads, head_dim // 16, KV_PAGE, 16),
                   new(num_pages, num_heads, head_dim, KV_PAGE), new(num_pages, num_heads),
                   new(num_pages, num_heads))


def kv_cache_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, row_offsets: torch.Tensor,
                    kv_lens: torch.Tensor, block_table: torch.Tensor, max_new: int, stream=None):
    """Write new tokens: rows row_offsets[s] .. row_offsets[s + 1] of ``k`` and
    ``v`` (BF16 [rows, heads, D]) are the last tokens of sequence s, whose
    length ``kv_lens`` counts them.  ``max_new`` bounds a sequence's rows."""
    _serving.append(cache, k, v, row_offsets, block_table, kv_lens, max_new, stream)


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
    r = _serving.attention(q, cache, row_offsets, block_table, kv_lens, max_q, max_kv,
                           q.shape[-1] ** -0.5 if scale is None else scale, window, out, lse,
                           return_lse, workspace, 0, None, stream)
    return r if return_lse else r[0]


def kv_pages_copy(cache: KvCache, src: torch.Tensor, dst: torch.Tensor, stream=None):
    """Page dst[i] becomes a copy of page src[i] (int32 vectors; distinct
    destinations, none of them a source of another pair)."""
    _serving.pages_copy(cache, src, dst, stream)


def kv_pages_reserve(block_table: torch.Tensor, kv_lens: torch.Tensor, refcounts: torch.Tensor,
                     slots: torch.Tensor, add_tokens: torch.Tensor, status=None, stream=None):
    """Lengthen sequences slots[i] by add_tokens[i] tokens, with pages of
    refcount 0, lowest number first, requests in order.  Returns status
    (int32: 0 done, 1 no pages or table entries left, 2 no such slot).  To take
    tokens back, lower ``kv_lens``, after taking 1 off the ``refcounts`` of the
    pages at the row's end that this gives up; the page that it ends in must be
    the sequence's own (``include/bsq_serving.h``)."""
    return _serving.pages_reserve(block_table, kv_lens, refcounts, slots, add_tokens, status,
                                  stream)


def kv_pages_fork(cache: KvCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                  refcounts: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
                  status=None, stream=None):
    """Slot children[i] (empty) becomes a copy of slot parents[i]: full pages
    shared, a partly filled last page copied.  Returns status as
    ``kv_pages_reserve`` does."""
    return _serving.pages_fork(cache, block_table, kv_lens, refcounts, parents, children, status,
                               stream)


def kv_pages_free(block_table: torch.Tensor, kv_lens: torch.Tensor, refcounts: torch.Tensor,
                  slots: torch.Tensor, stream=None):
    """Sequences slots[i] give their pages back and get length 0."""
    _serving.pages_free(block_table, kv_lens, refcounts, slots, stream)


def kv_pages_compact(cache: KvCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                     refcounts: torch.Tensor, table_out=None, refcounts_out=None, num_live=None,
                     workspace=None, stream=None):
    """Move the pages in use to the front of the cache.  Returns (table,
    refcounts, num_live int32 [1]); the outputs may be the inputs themselves
    (``table_out=block_table``, ``refcounts_out=refcounts``)."""
    return _serving.pages_compact(cache, block_table, kv_lens, refcounts, table_out, refcounts_out,
                                  num_live, workspace, stream)


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
    return _serving.moe(x, _fmt(fmt), w13_codes, w13_scales, w2_codes, w2_scales, num_experts, topk,
                        router_logits, topk_ids, topk_weights, renormalize, out, workspace, stream)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                 v=None, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None, v_out=None, stream=None):
    """Norms of queries and keys for each head and their rotation by position.
    ``q`` and ``k`` [rows, heads, D], BF16 or both FP32 (slices of one
    projection's output do); with ``q_weight`` / ``k_weight`` (fp32 [D])
    x * weight / sqrt(mean x^2 + eps), then the first 2 * len(inv_freq)
    elements of a head turned by positions (int32 [rows]) * inv_freq (float64,
    radians a token): pairs (i, i + len), or neighbours with ``interleaved``.
    Returns BF16 (q, k, v): v is rounded only, None where none is given.  An
    output may be its BF16 input itself."""
    return _serving.rope(q, k, v, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out,
                         k_out, v_out, stream)


def kv_cache_attention_masked(q: torch.Tensor, cache: KvCache, row_offsets: torch.Tensor,
                              kv_lens: torch.Tensor, block_table: torch.Tensor, max_q: int,
                              max_kv: int, masks=None, sinks: int = 0, scale: float | None = None,
                              window: int = 0, out=None, return_lse: bool = False, lse=None,
                              workspace=None, stream=None):
    """``kv_cache_attention`` with two more masks.  ``sinks``: with a window,
    that many first tokens of a sequence stay visible.  ``masks`` (int64 or
    uint64 [rows, words]): the rows are nodes of a tree of drafted tokens, and
    a row sees those rows of its sequence whose bits (x % 64 of word x / 64)
    are set, itself only if its own is, beside the tokens before them; a window
    counts the rows seen.  All else as there."""
    r = _serving.attention(q, cache, row_offsets, block_table, kv_lens, max_q, max_kv,
                           q.shape[-1] ** -0.5 if scale is None else scale, window, out, lse,
                           return_lse, workspace, sinks, masks, stream)
    return r if return_lse else r[0]


SCORES = {"softmax": 0, "sigmoid": 1}


def moe_route(logits: torch.Tensor, topk: int, score: str = "softmax", bias=None,
              num_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
              renormalize: bool = True, factor: float = 1.0, topk_ids=None, topk_weights=None,
              stream=None):
    """Experts of each token from a router's ``logits`` (BF16 or FP32 [tokens,
    experts]): scores by ``score`` ("softmax" or "sigmoid"), the ``topk``
    largest of score + ``bias`` (fp32 [experts]) among the ``topk_groups`` of
    ``num_groups`` groups whose ``group_top`` (1 or 2) largest have the largest
    sum.  Weights are ``factor`` times the scores, divided by the sum of the
    chosen ones with ``renormalize``.  The choice is that of 64-bit arithmetic,
    ties to the lower number.  Returns (topk_ids int32, topk_weights fp32)
    [tokens, topk], as ``moe_few_tokens`` takes them."""
    if score not in SCORES:
        raise BsqError(2, f"score={score!r} is not provided (softmax or sigmoid)")
    return _serving.route(logits, topk, SCORES[score], bias, num_groups, topk_groups, group_top,
                          renormalize, factor, topk_ids, topk_weights, stream)


def moe_group_rows(topk_ids: torch.Tensor, num_experts: int, pad: int = 128, row_offsets=None,
                   scales_offsets=None, row_indices=None, entry_rows=None, workspace=None,
                   stream=None):
    """The routed rows of each expert for the grouped quantizer and GEMM, from
    ``topk_ids`` (int32 [tokens, topk]; numbers outside the experts have no
    row), an expert's entries in their order.  Returns int32 (row_offsets
    [experts + 1], scales_offsets [experts + 1], a group's scale rows being
    its rows rounded up to a multiple of ``pad``, row_indices [tokens * topk],
    the token of each routed row or -1 past the last, entry_rows [tokens, topk],
    the routed row of each entry or -1)."""
    return _serving.group_rows(topk_ids, num_experts, pad, row_offsets, scales_offsets, row_indices,
                               entry_rows, workspace, stream)


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` gives: the log probabilities of the given tokens
    (fp32, their shape; None without any), each row's entropy (fp32 [rows]) and
    its likeliest tokens, the likeliest first (int32 and fp32 [rows, top])."""
    logprobs: torch.Tensor | None
    entropy: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor


def token_logprobs(logits: torch.Tensor, tokens=None, top: int = 0, workspace=None,
                   stream=None) -> TokenLogprobs:
    """Log probabilities of ``tokens`` (int32 [rows] or [rows, n]) under
    softmax(``logits``) (BF16 or FP32 [rows, vocab]), the entropy of each row
    and its ``top`` likeliest tokens (up to 64; equal ones by their number), in
    one pass over the logits.  A token outside the vocabulary has -inf."""
    return TokenLogprobs(*_serving.logprobs(logits, tokens, top, workspace, stream))
