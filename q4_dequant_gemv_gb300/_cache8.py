"""The paged cache in 8 bits and what stands beside it: q4k_norm_rope, q4k_kv_append8, q4k_kv_read8 and
q4k_paged_attention8 (include/q4k.h says what each computes; csrc/q4k_marshal.c checks their arguments and calls the library).

An 8-bit cache is k_cache, v_cache [pages, page size, heads, dim] of codes, int8 or float8_e4m3fn (any strides), and
k_scale, v_scale fp32 [pages, blocks of a page, heads] (any strides): a block is page size / blocks consecutive slots, a
power of two up to 128, and a cached value is its code times its block's scale.  Blocks of one token never change their
scale; larger ones take less memory and share their largest value."""
from __future__ import annotations

import ctypes

import torch

from . import _attention

_calls = None


def _load():
    """The compiled calls (there is no fallback path)."""
    global _calls
    from . import lib
    m = _attention._calls or _attention._load()
    L = lib()
    m.setup8(torch.int8, torch.float8_e4m3fn, *(ctypes.cast(f, ctypes.c_void_p).value
                                                for f in (L.q4k_norm_rope, L.q4k_kv_append8, L.q4k_kv_read8,
                                                          L.q4k_paged_attention8)))
    _calls = m
    return m


def norm_rope(q, k=None, pos=None, table=None, q_weight=None, k_weight=None, q_out=None, k_out=None, *, eps: float = 1e-6,
              interleaved: bool = False, out_dtype=None, stream=None, pdl: bool = False):
    """(q_out, k_out): each head of q and k [tokens, heads, dim] over its root mean square (with eps under the root) times
    its weight, fp32 [dim] or [heads, dim] (None: as it is), then turned as rope turns it by row pos[token] of the table
    (None: not turned).  k may be None; q_out and k_out may be q and k themselves."""
    return (_calls or _load()).norm_rope(q, k, pos, table, q_weight, k_weight, q_out, k_out, eps, interleaved, out_dtype, stream,
                                         pdl)


def kv_append8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, *, table=None, interleaved: bool = False,
               pos=None, q=None, q_out=None, q_dtype=None, q_weight=None, k_weight=None, eps: float = 1e-6, stream=None,
               pdl: bool = False):
    """kv_append into an 8-bit cache: keys normed (k_weight) and turned, values as they are, quantised with a scale for each
    block and head.  A block that already holds older tokens of its sequence keeps its scale, or takes a larger one and
    has the older codes rounded again.  Queries, where given, are normed (q_weight) and turned into q_out.  Caches or scales
    that repeat themselves (a stride of 0) are refused."""
    return (_calls or _load()).kv_append8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, table,
                                          interleaved, pos, q, q_out, q_dtype, q_weight, k_weight, eps, stream, pdl)


def kv_read8(k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, tokens: int, k=None, v=None, *, dtype=None,
             stream=None, pdl: bool = False):
    """(k, v) [tokens, heads, dim]: the cached values of the last seq_start[b + 1] - seq_start[b] positions of each sequence
    (those that kv_append8 with the same arrays writes; all of them where seq_start counts up kv_len), in dtype (bfloat16
    unless given).  tokens: rows of the outputs; those of no sequence are left as they are."""
    if dtype is None:
        dtype = next((t.dtype for t in (k, v) if t is not None), torch.bfloat16)
    return (_calls or _load()).kv_read8(k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, tokens, k, v, dtype,
                                        stream, pdl)


def paged_attention8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, out=None, *, scale=None,
                     out_dtype=None, softcap: float = 0.0, slopes=None, window: int = 0, causal: bool = True, prefix_len=None,
                     kv_start=None, lse=None, stream=None, pdl: bool = False, wait_limit_us: int = 0, test_stall: bool = False,
                     form=None):
    """paged_attention over an 8-bit cache (all options as there; dim a multiple of 16).  Prompt chunks take scratch as wide as
    the page table (scratch_keep says how much of it stays)."""
    if form not in _attention._FORMS:
        raise ValueError(f"form must be one of {list(_attention._FORMS)}")
    return (_calls or _load()).paged_attention8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, out, scale,
                                                out_dtype, softcap, slopes, window, causal, prefix_len, kv_start, lse, stream,
                                                (1 if pdl else 0) | (8 if test_stall else 0) | _attention._FORMS[form] << 8,
                                                wait_limit_us)
