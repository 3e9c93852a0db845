"""Rotary positions, the paged cache and attention over it: q4k_rope_table, q4k_rope, q4k_kv_append and
q4k_paged_attention (include/q4k.h says what each computes).  Argument marshalling only, like the rest of the
binding; these calls sit between a layer's products, so their structures are packed in one go."""
from __future__ import annotations

import math
import struct

import torch

Q4K_F32, Q4K_F16, Q4K_BF16 = 0, 1, 2
_CODE = {torch.float32: Q4K_F32, torch.float16: Q4K_F16, torch.bfloat16: Q4K_BF16}
_SCALING = {None: 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}

# The C structures, field by field (native alignment).
_ROPE = struct.Struct("@4P 5q 4q 4i")
_SCALE = struct.Struct("@6d 2i")
_CACHE = struct.Struct("@2P 6q 4q P 2q 2P 2q 2i")
_APPEND = struct.Struct("@4P 8q 2P 3q 6i")
_ATTENTION = struct.Struct("@3P 4q 2q 3P 2f 6i")


_lib = None
# The handle of a device's current stream, without building a Stream object around it (3 us a call).
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _load():
    global _lib
    from . import lib
    _lib = lib()
    return _lib


def _raise(fn, status):
    from . import _check
    _check(fn, status)


def _stream(stream, t):
    return _current(t.get_device()) if stream is None else stream.cuda_stream


# (What follows runs between a decode step's launches: attributes are read once, and
# tensors made here are not checked again.)
_Tensor = torch.Tensor
_i32 = torch.int32


def _rows(t, name, heads=None, dim=None, tokens=None):
    """Address, type code, shape and strides of a [tokens, heads, dim] tensor."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], got {tuple(shape)}")
    n, h, d = shape
    if (heads is not None and h != heads) or (dim is not None and d != dim) or (tokens is not None and n != tokens):
        want = ", ".join("*" if v is None else str(v) for v in (tokens, heads, dim))
        raise ValueError(f"{name} must be [{want}], got {tuple(shape)}")
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr(), code, n, h, d, st, sh


def _array(t, name, dtype, n):
    """Address of a contiguous device array of n values."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous array of {n}, got {tuple(t.shape)}")
    return t.data_ptr()


def _turn(table, rot_max):
    """Address, rows and rot of a rotary table (None: no rotation)."""
    if table is None:
        return 0, 0, 0
    if not isinstance(table, _Tensor):
        raise TypeError("table must be a torch.Tensor")
    if table.dtype is not torch.float32:
        raise TypeError(f"table must have dtype torch.float32, got {table.dtype}")
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    shape = table.shape
    if len(shape) != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous [positions, rot] tensor")
    rows, rot = shape
    if rot % 2 or rot > rot_max:
        raise ValueError(f"table turns {rot} of {rot_max} elements of a head")
    return table.data_ptr(), rows, rot


def _cache(k_cache, v_cache, page_table, seq_start, kv_len, tokens):
    """The packed q4k_paged_cache, its heads, dim and sequences."""
    if not (isinstance(k_cache, _Tensor) and isinstance(v_cache, _Tensor) and isinstance(page_table, _Tensor)):
        raise TypeError("k_cache, v_cache and page_table must be torch.Tensors")
    if not (k_cache.is_cuda and v_cache.is_cuda and page_table.is_cuda):
        raise ValueError("k_cache, v_cache and page_table must be CUDA tensors")
    dtype, shape = k_cache.dtype, k_cache.shape
    code = _CODE.get(dtype)
    if not code:      # (fp32 is 0)
        raise TypeError(f"k_cache must be bfloat16 or float16, got {dtype}")
    if v_cache.dtype is not dtype:
        raise TypeError(f"v_cache must have dtype {dtype}, got {v_cache.dtype}")
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache and v_cache must be [pages, page size, heads, dim], got {tuple(shape)} and "
                         f"{tuple(v_cache.shape)}")
    pages, size, heads, dim = shape
    kp, ks, kh, kd = k_cache.stride()
    vp, vs, vh, vd = v_cache.stride()
    if (kd != 1 or vd != 1) and dim > 1:
        raise ValueError("k_cache and v_cache must be contiguous in their last dimension")
    if page_table.dtype is not _i32:
        raise TypeError(f"page_table must have dtype torch.int32, got {page_table.dtype}")
    table = page_table.shape
    if len(table) != 2:
        raise ValueError(f"page_table must be [sequences, pages], got {tuple(table)}")
    batch, most = table
    row, step = page_table.stride()
    if step != 1 and most > 1:
        raise ValueError("page_table must be contiguous in its last dimension")
    packed = _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), kp, ks, kh, vp, vs, vh, pages, size, heads, dim,
                         page_table.data_ptr(), row, most, _array(seq_start, "seq_start", _i32, batch + 1),
                         _array(kv_len, "kv_len", _i32, batch), batch, tokens, code, 0)
    return packed, heads, dim, batch


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
        table = torch.empty((rows, rot), dtype=torch.float32, device=device)
        args = _SCALE.pack(base, factor, orig_len, low, high, magnitude, _SCALING[scaling], 0)
        st = (_lib or _load()).q4k_rope_table(table.data_ptr(), rows, rot, args, _stream(stream, table))
        if st:
            _raise("q4k_rope_table", st)
        if stream is not None:
            table.record_stream(stream)
    return table


def _new(like, dtype, shape, stream):
    """Address and type code of a new tensor that the call's stream may use."""
    t = torch.empty_like(like) if dtype is like.dtype and like.is_contiguous() else torch.empty(shape, dtype=dtype, device=like.device)
    if stream is not None:
        t.record_stream(stream)
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError(f"the output must be float32, float16 or bfloat16, got {dtype}")
    return t, t.data_ptr(), code


def rope(x, pos, table, y=None, *, interleaved: bool = False, out_dtype=None, stream=None,
         pdl: bool = False):
    """y [tokens, heads, dim] = x with the first table.shape[1] elements of each head turned by row pos[token] of the
    table; pairs (i, i + rot/2), or (2i, 2i+1) if interleaved.  y may be x."""
    xp, xc, n, h, d, xt, xh = _rows(x, "x")
    tp, rows, rot = _turn(table, d)
    if pos is None and rot:
        raise ValueError("pos is needed with a table")
    pp = 0 if pos is None else _array(pos, "pos", _i32, n)
    if y is None:
        y, yp, yc = _new(x, out_dtype or x.dtype, (n, h, d), stream)
        yt, yh = h * d, d
    else:
        yp, yc, _, _, _, yt, yh = _rows(y, "y", h, d, n)
        if out_dtype is not None and y.dtype is not out_dtype:
            raise TypeError(f"y must have dtype {out_dtype}, got {y.dtype}")
    args = _ROPE.pack(xp, yp, pp, tp, n, h, d, rot, rows, xt, xh, yt, yh, xc, yc, 1 if interleaved else 0, 1 if pdl else 0)
    st = (_lib or _load()).q4k_rope(args, _stream(stream, x))
    if st:
        _raise("q4k_rope", st)
    return y


def kv_append(k, v, k_cache, v_cache, page_table, seq_start, kv_len, *, table=None, interleaved: bool = False, pos=None,
              q=None, q_out=None, q_dtype=None, stream=None, pdl: bool = False):
    """Stores the new tokens' keys (turned by the table) and values [tokens, heads, dim] in the paged cache
    [pages, page size, heads, dim] (any strides).  Rows seq_start[b] .. seq_start[b+1]-1 are the last new tokens of
    sequence b, whose cache holds kv_len[b] positions with them.  q [tokens, q heads, dim], where given, is turned too:
    returns q_out (of q_dtype, or q's type), else None."""
    kp, kc, n, h, d, kt, kh = _rows(k, "k")
    vp, vc, _, _, _, vt, vh = _rows(v, "v", h, d, n)
    if vc != kc:
        raise TypeError("k and v must have the same dtype")
    cache, ch, cd, _ = _cache(k_cache, v_cache, page_table, seq_start, kv_len, n)
    if ch != h or cd != d:
        raise ValueError(f"the cache holds {ch} heads of {cd}, k and v {h} of {d}")
    tp, rows, rot = _turn(table, d)
    pp = 0 if pos is None else _array(pos, "pos", _i32, n)
    qp = qc = qh = qts = qhs = op = oc = ots = ohs = 0
    if q is not None:
        qp, qc, _, qh, _, qts, qhs = _rows(q, "q", None, d, n)
        if q_out is None:
            q_out, op, oc = _new(q, q_dtype or q.dtype, (n, qh, d), stream)
            ots, ohs = qh * d, d
        else:
            op, oc, _, _, _, ots, ohs = _rows(q_out, "q_out", qh, d, n)
            if q_dtype is not None and q_out.dtype is not q_dtype:
                raise TypeError(f"q_out must have dtype {q_dtype}, got {q_out.dtype}")
    elif q_out is not None:
        raise ValueError("q_out without q")
    args = _APPEND.pack(kp, vp, qp, op, kt, kh, vt, vh, qts, qhs, ots, ohs, pp, tp, rows, rot, qh, kc, qc, oc,
                        1 if interleaved else 0, 1 if pdl else 0, 0)
    st = (_lib or _load()).q4k_kv_append(cache, args, _stream(stream, k))
    if st:
        _raise("q4k_kv_append", st)
    return q_out


def paged_attention(q, k_cache, v_cache, page_table, seq_start, kv_len, out=None, *, scale=None, out_dtype=None,
                    softcap: float = 0.0, slopes=None, window: int = 0, causal: bool = True, prefix_len=None,
                    kv_start=None, lse=None, stream=None, pdl: bool = False, wait_limit_us: int = 0,
                    test_stall: bool = False):
    """out [tokens, q heads, dim] = attention of the new tokens over their sequences' cached positions, the new ones
    included (the cache, seq_start and kv_len as kv_append leaves them).  Token t at position p sees
    max(0, kv_start[t], p + 1 - window) <= j < max(p + 1, prefix_len[b]), or < kv_len[b] if not causal.
    scale: 1/sqrt(dim) unless given; softcap > 0: scores softcap * tanh(s / softcap); slopes fp32 [q heads]: minus
    slopes[h] * |p - j|; lse: fp32 [tokens, q heads], filled with the rows' log-sum-exp.  wait_limit_us, test_stall:
    bound of the kernel's waits, and a wait made to run out (failure tests)."""
    qp, qc, n, h, d, qt, qh = _rows(q, "q")
    cache, ch, cd, batch = _cache(k_cache, v_cache, page_table, seq_start, kv_len, n)
    if cd != d or ch < 1 or h % ch:
        raise ValueError(f"the cache holds {ch} heads of {cd}, q {h} of {d}")
    if out is None:
        out, op, oc = _new(q, out_dtype or q.dtype, (n, h, d), stream)
        ot, oh = h * d, d
    else:
        op, oc, _, _, _, ot, oh = _rows(out, "out", h, d, n)
        if out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out must have dtype {out_dtype}, got {out.dtype}")
    lp = 0
    if lse is not None:
        if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32:
            raise TypeError("lse must be a float32 tensor")
        if not lse.is_cuda or not lse.is_contiguous() or tuple(lse.shape) != (n, h):
            raise ValueError(f"lse must be a contiguous CUDA tensor [{n}, {h}]")
        lp = lse.data_ptr()
    args = _ATTENTION.pack(qp, op, lp, qt, qh, ot, oh, h, window,
                           0 if slopes is None else _array(slopes, "slopes", torch.float32, h),
                           0 if prefix_len is None else _array(prefix_len, "prefix_len", _i32, batch),
                           0 if kv_start is None else _array(kv_start, "kv_start", _i32, n),
                           1.0 / math.sqrt(d) if scale is None else scale, softcap, qc, oc, 1 if causal else 0,
                           (1 if pdl else 0) | (8 if test_stall else 0), wait_limit_us, 0)
    st = (_lib or _load()).q4k_paged_attention(cache, args, _stream(stream, q))
    if st:
        _raise("q4k_paged_attention", st)
    return out
