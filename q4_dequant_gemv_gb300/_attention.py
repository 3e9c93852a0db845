"""Rotary positions, the paged cache and attention over it: q4k_rope_table, q4k_rope, q4k_kv_append and
q4k_paged_attention (include/q4k.h says what each computes).  The last three sit between the launches of a decode
step; csrc/q4k_marshal.c checks their arguments and calls the library."""
from __future__ import annotations

import ctypes
import math
import struct

import torch

_SCALING = {None: 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}
_FORMS = {None: 0, "cluster8": 1, "cluster16": 2, "cluster32": 3, "split8": 4, "split16": 5, "split32": 6, "many": 7}
_SCALE = struct.Struct("@6d 2i")      # q4k_rope_scaling

# The handle of a device's current stream, without building a Stream object around it (3 us a call).
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
# The current device, likewise.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_calls = None


def _new_on(stream, shape, dtype, device):
    """A new tensor that a given stream writes: from that stream's own blocks.  One that the current stream has freed may
    still be read there, and nothing orders the two.  The current stream, which may go on with the tensor, is recorded."""
    now = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(now)
    return t


def _raise(fn, status):
    from . import _check
    _check(fn, status)


def _load():
    """The compiled calls (there is no fallback path)."""
    global _calls
    from . import lib
    L = lib()
    try:
        from . import _marshal
    except ImportError as e:
        raise RuntimeError("the _marshal module is not built; run __graft_entry__.build()") from e
    _marshal.setup(torch.Tensor, torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.empty, torch.empty_like,
                   _new_on, _device, _current, _raise, *(ctypes.cast(f, ctypes.c_void_p).value for f in
                                       (L.q4k_rope, L.q4k_kv_append, L.q4k_paged_attention)))
    _calls = _marshal
    return _marshal


def rope_table(rows: int, rot: int, base: float = 10000.0, *, scaling=None, factor: float = 1.0, orig_len: float = 0.0,
               low=None, high=None, magnitude=None, device=None, stream=None):
    """fp32 [rows, rot]: cosines and sines of positions 0 .. rows-1, the angles formed in 64 bits.
    scaling: None, "linear" (positions divided by factor), "base" (the base grows with factor), "ramp" (slow pairs
    interpolated, fast ones kept, a ramp between the pairs that turn `low` and `high` times over orig_len positions:
    1 and 32 unless given; magnitude 0.1 ln(factor) + 1 unless given) or "bands" (the same by wavelength: 1 and 4)."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling must be one of {list(_SCALING)}")
    low = 1.0 if low is None else low
    high = (4.0 if scaling == "bands" else 32.0) if high is None else high
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "ramp" and factor > 1 else 1.0
    if rows < 0 or rot < 2 or rot % 2:
        raise ValueError(f"bad table {rows} x {rot}")
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        table = (torch.empty((rows, rot), dtype=torch.float32, device=device) if stream is None
                 else _new_on(stream, (rows, rot), torch.float32, device))
        from . import _check, lib
        args = _SCALE.pack(base, factor, orig_len, low, high, magnitude, _SCALING[scaling], 0)
        on = _current(table.get_device()) if stream is None else stream.cuda_stream
        _check("q4k_rope_table", lib().q4k_rope_table(table.data_ptr(), rows, rot, args, on))
    return table


def rope(x, pos, table, y=None, *, interleaved: bool = False, out_dtype=None, stream=None,
         pdl: bool = False):
    """y [tokens, heads, dim] = x with the first table.shape[1] elements of each head turned by row pos[token] of the
    table; pairs (i, i + rot/2), or (2i, 2i+1) if interleaved.  y may be x."""
    return (_calls or _load()).rope(x, pos, table, y, interleaved, out_dtype, stream, pdl)


def kv_append(k, v, k_cache, v_cache, page_table, seq_start, kv_len, *, table=None, interleaved: bool = False, pos=None,
              q=None, q_out=None, q_dtype=None, stream=None, pdl: bool = False):
    """Stores the new tokens' keys (turned by the table) and values [tokens, heads, dim] in the paged cache
    [pages, page size, heads, dim] (any strides).  Rows seq_start[b] .. seq_start[b+1]-1 are the last new tokens of
    sequence b, whose cache holds kv_len[b] positions with them.  q [tokens, q heads, dim], where given, is turned too:
    returns q_out (of q_dtype, or q's type), else None."""
    return (_calls or _load()).kv_append(k, v, k_cache, v_cache, page_table, seq_start, kv_len, table, interleaved, pos, q,
                                         q_out, q_dtype, stream, pdl)


def paged_attention(q, k_cache, v_cache, page_table, seq_start, kv_len, out=None, *, scale=None, out_dtype=None,
                    softcap: float = 0.0, slopes=None, window: int = 0, causal: bool = True, prefix_len=None,
                    kv_start=None, lse=None, stream=None, pdl: bool = False, wait_limit_us: int = 0,
                    test_stall: bool = False, form=None):
    """out [tokens, q heads, dim] = attention of the new tokens over their sequences' cached positions, the new ones
    included (the cache, seq_start and kv_len as kv_append leaves them).  Token t at position p sees
    max(0, kv_start[t], p + 1 - window) <= j < max(p + 1, prefix_len[b]), or < kv_len[b] if not causal.
    scale: 1/sqrt(dim) unless given; softcap > 0: scores softcap * tanh(s / softcap); slopes fp32 [q heads]: minus
    slopes[h] * |p - j|; lse: fp32 [tokens, q heads], filled with the rows' log-sum-exp.  wait_limit_us, test_stall:
    bound of the kernel's waits, and a wait made to run out (failure tests).  form: one form of the kernels, "cluster8"
    .. "many", instead of the library's choice by sizes."""
    if form not in _FORMS:
        raise ValueError(f"form must be one of {list(_FORMS)}")
    return (_calls or _load()).paged_attention(q, k_cache, v_cache, page_table, seq_start, kv_len, out, scale, out_dtype,
                                               softcap, slopes, window, causal, prefix_len, kv_start, lse, stream,
                                               (1 if pdl else 0) | (8 if test_stall else 0) | _FORMS[form] << 8,
                                               wait_limit_us)
