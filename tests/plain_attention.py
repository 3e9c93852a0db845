"""Rotary positions, paged append and paged attention in 64 bits, straight from their definitions, with the error
bounds that the kernels' arithmetic allows.  CPU only; shared by the tests of those operators."""
import math

import torch

# unit roundoff of the types (half an ulp of 1)
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half of the smallest subnormal step
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


def table(rows, rot, base=10000.0, factor=1.0):
    """fp32 [rows, rot] of cosines and sines of p / factor * base^(-2i/rot)."""
    f = torch.tensor([base ** (-2.0 * i / rot) / factor for i in range(rot // 2)], dtype=torch.float64)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def turn(x, rows, interleaved):
    """x [tokens, heads, dim] turned by the table rows [tokens, rot], in 64 bits; and the sum of |terms|."""
    x, rows = x.double(), rows.double()
    rot = rows.shape[1]
    y, mag = x.clone(), x.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = rows[:, i][:, None], rows[:, rot // 2 + i][:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., a] * s).abs() + (x[..., b] * c).abs()
    return y, mag


def turn_bound(y, mag, dtype):
    """Two products and a sum in fp32 (three roundings of at most 2^-24 of the terms), one rounding to dtype."""
    return 4 * 2.0 ** -24 * mag + UNIT[dtype] * (y.abs() + 4 * 2.0 ** -24 * mag) + TINY[dtype]


def ranges(case):
    """[(sequence, position, lo, hi)] of every token."""
    out = []
    for b, (n, length) in enumerate(zip(case["new"], case["len"])):
        for i in range(n):
            p = length - n + i
            hi = length
            if case.get("causal", True):
                hi = p + 1
                if case.get("prefix") is not None:
                    hi = max(hi, case["prefix"][b])
                hi = max(0, min(hi, length))
            lo = 0
            if case.get("window"):
                lo = max(lo, p + 1 - case["window"])
            if case.get("kv_start") is not None:
                lo = max(lo, case["kv_start"][len(out)])
            out.append((b, p, lo, max(lo, hi)))
    return out


def attention(q, keys, values, case, scale, softcap=0.0, slopes=None, parts=True, cache_dtype=torch.bfloat16,
              out_dtype=torch.float32):
    """out, lse and the bound of |out - kernel's| per element.  keys, values: per sequence [len, kv heads, dim].

    The bound: with e the error of a score (fp32 accumulation of dim products on the tensor cores, taken as
    dim 2^-23 of sum |q k|; its scaling, cap and distance terms; the parts of an fp32 q), every weight is off by at
    most 2 e + 2^-20 of itself, and by the cache type's unit where it is rounded once; sums of L terms by
    (16 + sqrt L) 2^-22; the output by its type's unit."""
    T, H, D = q.shape
    out = torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    bound = torch.zeros(T, H, D, dtype=torch.float64)
    qd = q.double()
    for t, (b, p, lo, hi) in enumerate(ranges(case)):
        if hi <= lo:
            continue
        g = H // keys[b].shape[1]
        k, v = keys[b][lo:hi].double(), values[b][lo:hi].double()
        k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)          # [L, H, D]
        s = torch.einsum("hd,jhd->hj", qd[t], k) * scale
        size = torch.einsum("hd,jhd->hj", qd[t].abs(), k.abs()) * abs(scale)
        e = (D + 8) * 2.0 ** -23 * size.amax(1) + 2.0 ** -21 * s.abs().amax(1)
        if parts:
            e = e + 2.0 ** -21 * size.amax(1)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            e = e + softcap * 2.0 ** -20
        if slopes is not None:
            away = (p - torch.arange(lo, hi, dtype=torch.float64)).abs()
            s = s - slopes.double()[:, None] * away
            e = e + 2.0 ** -21 * slopes.double().abs() * away.max()
        lse[t] = torch.logsumexp(s, 1)
        w = torch.softmax(s, 1)
        out[t] = torch.einsum("hj,jhd->hd", w, v)
        mag = torch.einsum("hj,jhd->hd", w, v.abs())
        rel = 2 * e + 2.0 ** -20 + (0.0 if parts else UNIT[cache_dtype]) + (16 + math.sqrt(hi - lo)) * 2.0 ** -22
        bound[t] = rel[:, None] * mag
    bound = bound + UNIT[out_dtype] * (out.abs() + bound) + TINY[out_dtype]
    return out, lse, bound


def paged(seqs, page_size, dtype, order, spare=2, fill=float("nan"), heads_first=False):
    """(cache, page_table): the sequences [len, heads, dim] laid out in pages taken in the given random order, every
    slot that holds no position filled with `fill`, unused table entries -1."""
    counts = [-(-s.shape[0] // page_size) for s in seqs]
    h, d = seqs[0].shape[1:]
    n = sum(counts) + spare
    cache = torch.full((n, page_size, h, d), fill, dtype=dtype)
    perm = order[order < n].tolist()
    pt = torch.full((len(seqs), max(counts + [1])), -1, dtype=torch.int32)
    at = 0
    for b, s in enumerate(seqs):
        for i in range(counts[b]):
            pg = perm[at]
            at += 1
            pt[b, i] = pg
            part = s[i * page_size:(i + 1) * page_size]
            cache[pg, :part.shape[0]] = part.to(dtype)
    if heads_first:
        cache = cache.transpose(1, 2).contiguous().transpose(1, 2)
    return cache, pt
