"""Attention over an 8-bit paged cache where much of the cache is seen by nobody: tiles that see nothing at all, scales
of slots that no token sees, before its keys or between them.  All forms of the kernels."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402
from test_attention8_gpu import (BF16, E4M3, F16, F32, FORMS, I8, _cache, _dev, _floor, _products, _takes, q4k)   # noqa: E402,F401

pytestmark = pytest.mark.gpu
NOTHING = 10 ** 9


def _starts(new):
    return _dev([sum(new[:i]) for i in range(len(new) + 1)])


def _options(case):
    return dict(window=case.get("window", 0), causal=case.get("causal", True),
                prefix_len=None if case.get("prefix") is None else _dev(case["prefix"]),
                kv_start=None if case.get("kv_start") is None else _dev(case["kv_start"]))


def _check(out, lse, q, keys, vals, vs, vc, case, form, page):
    """out and lse against 64 bits; rows that see nothing are zero, their log-sum-exp -inf."""
    qt, D = q.dtype, q.shape[2]
    many = qt != F32 and D <= 128 and page % 16 == 0 and form in (None, "many")
    ref, rl, bound = plain.attention(q, keys, vals, case, 1.0 / math.sqrt(D), 0.0, None, qt == F32, F16, qt)
    more, off = _products(q, keys, vals, case, 1.0 / math.sqrt(D), None, 0.0) if many else (0.0, torch.zeros_like(rl))
    bound = bound + _floor(vs, vc, case["len"], many) + more
    assert ((out.double().cpu() - ref).abs() <= bound).all()
    dead = torch.isinf(rl)
    got = lse.double().cpu()
    assert torch.equal(dead, torch.isinf(got) & (got < 0)) and not out.cpu()[dead].any()
    assert ((got[~dead] - rl[~dead]).abs() <= 2.0 ** -12 + 2.0 ** -20 * rl[~dead].abs() + off[~dead]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("qt,ct,block", [(BF16, I8, 16), (F16, E4M3, 16), (BF16, E4M3, 4), (F16, I8, 64), (F32, I8, 16)])
@pytest.mark.parametrize("case", [
    # the last sequence's tokens start behind its keys, the table ends with them
    dict(new=[4, 40], len=[130, 300], kv_start=[0] * 4 + [NOTHING] * 40),
    dict(new=[40, 300], len=[300, 384], kv_start=[300] * 40 + [384] * 300),
    # nothing is cached, beside a sequence that has something; a whole tile of padding between tokens that see
    dict(new=[5, 33], len=[200, 0]),
    dict(new=[3, 0, 70], len=[0, 0, 100], window=9),
    dict(new=[300], len=[512], kv_start=[0] * 40 + [NOTHING] * 220 + [500] * 40),
    dict(new=[20, 300], len=[40, 400], causal=False, kv_start=[NOTHING] * 20 + [390] * 10 + [400] * 290),
], ids=range(6))
def test_tiles_that_see_nothing(q4k, case, qt, ct, block, form):   # noqa: F811
    """Zeros and -inf for rows that see nothing, whatever an earlier call left in the scratch, and the other rows as ever."""
    H, KH, D, page = 4, 2, 64, 64
    if not _takes(form, qt, qt, D, page, 1.0, 2, 0.0):
        return
    g = torch.Generator().manual_seed(sum(case["len"]) + block)
    ((kc, ks, keys), (vc, vs, vals)), pt = _cache(g, case["len"], page, block, KH, D, ct)
    q = (torch.randn(sum(case["new"]), H, D, generator=g, dtype=torch.float64) * 1.5).to(qt)
    start, pt = _starts(case["new"]), pt.cuda()
    # (an earlier call of the same size whose scales are infinite throughout)
    full = torch.full_like(ks, math.inf)
    q4k.paged_attention8(q.cuda(), kc, vc, full, full, pt.clamp(min=0), start, _dev([pt.shape[1] * page] * len(case["len"])), form=form)
    torch.cuda.synchronize()
    q4k.device_error_clear()
    lse = torch.full((q.shape[0], H), 7.0, device="cuda")
    out = q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, pt, start, _dev(case["len"]), lse=lse, form=form, **_options(case))
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    _check(out, lse, q, keys, vals, vs, vc, case, form, page)


@pytest.mark.parametrize("form", FORMS)
def test_lengths_past_the_table(q4k, form):   # noqa: F811
    """A window that lies behind the table's last page: flagged, nothing read there."""
    q = torch.ones(40, 2, 64, dtype=F16, device="cuda")
    kc, ks = torch.ones(9, 64, 1, 64, dtype=I8, device="cuda"), torch.ones(9, 4, 1, device="cuda")
    pt = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    for kw in (dict(window=5), dict(window=5, kv_start=_dev([NOTHING] * 40))):
        q4k.paged_attention8(q, kc, kc, ks, ks, pt, _dev([0, 20, 40]), _dev([500, 10 ** 6]), form=form, **kw)
        torch.cuda.synchronize()
        assert q4k.device_error_flags() == 4
        q4k.device_error_clear()


def _seen(case):
    """Which positions of each sequence some token sees."""
    seen = [torch.zeros(n, dtype=torch.bool) for n in case["len"]]
    for b, _, lo, hi in plain.ranges(case):
        seen[b][lo:hi] = True
    return seen


def _padded(n, length, seen, first=0):
    """kv_start of n new tokens: the ranges `seen` of them see the keys from `first` on (the first range) or from their range's
    own start on, the tokens between see nothing."""
    out, past = [NOTHING] * n, length - n
    for k, (a, b) in enumerate(seen):
        for i in range(a, b):
            out[i] = first if k == 0 else past + a
    return out


UNSEEN = {
    # keys that a sequence's every token starts behind: padding, what an engine has given up
    "padding": dict(new=[300, 3], len=[400, 90], kv_start=[40] * 300 + [70] * 3),
    "padding, no causal mask": dict(new=[20, 40], len=[300, 90], causal=False, kv_start=[150] * 20 + [33] * 40),
    # between documents, after tokens that see nothing
    "holes": dict(new=[200, 1, 64], len=[900, 20, 64],
                  kv_start=_padded(200, 900, [(0, 1), (60, 61), (150, 200)], 400) + [0] + _padded(64, 64, [(0, 3), (50, 64)])),
    "holes and a prefix": dict(new=[100], len=[400], prefix=[50], kv_start=_padded(100, 400, [(0, 1), (49, 50), (90, 100)])),
    "late": dict(new=[150], len=[400], kv_start=[250 + i + (1 if i % 50 > 16 else -(i % 50)) for i in range(150)]),
}
CASES = list(UNSEEN)
BLOCKS = [1, 4, 8, 16, 64]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("qt,ct", [(BF16, I8), (F16, E4M3), (F32, E4M3)])
@pytest.mark.parametrize("name,block", [(n, b) for n in CASES for b in BLOCKS])
def test_scales_that_nobody_sees(q4k, name, block, qt, ct, form):   # noqa: F811
    """Scales of slots that no token of the sequence sees, whatever they are: the bits that zeros there give."""
    case, H, KH, D, page = UNSEEN[name], 4, 2, 64, 64
    if not _takes(form, qt, qt, D, page, 1.0, 2, 0.0):
        return
    g = torch.Generator().manual_seed(sum(case["len"]) + block)
    ((kc, ks, keys), (vc, vs, vals)), pt = _cache(g, case["len"], page, block, KH, D, ct, spread=0.1)
    q = torch.randn(sum(case["new"]), H, D, generator=g).to(qt)
    args = (pt.cuda(), _starts(case["new"]), _dev(case["len"]))
    blocks = [(int(pt[b, p // page]), p % page // block) for b, s in enumerate(_seen(case)) for p in range(0, s.numel(), block)
              if not s[p:p + block].any()]
    if not blocks:
        return
    index = tuple(torch.tensor(x, device="cuda") for x in zip(*blocks))
    # a slot's codes of NaN and -128 too, where nobody sees it
    for b, s in enumerate(_seen(case)):
        p = (~s).nonzero()[:, 0]
        pages, slots = pt[b].long()[p // page].cuda(), (p % page).cuda()
        for c in (kc, vc):
            c.view(torch.uint8)[pages, slots] = 0x7F if ct == E4M3 else 0x80
    want = None
    for fill in (0.0, 1e30, math.inf, math.nan, -1e30):
        for s in (ks, vs):
            s[index] = fill
        lse = torch.full((q.shape[0], H), 7.0, device="cuda")
        out = q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, *args, lse=lse, form=form, **_options(case))
        torch.cuda.synchronize()
        assert q4k.device_error_flags() == 0
        if want is None:
            want = out, lse
            _check(out, lse, q, keys, vals, vs, vc, case, form, page)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), f"scales of {fill}: {float((out - want[0]).abs().max())} off"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("qt,ct", [(BF16, I8), (F16, E4M3), (F32, I8)])
@pytest.mark.parametrize("ratio", [0.0, 2.0 ** -45, 2.0 ** -33, 2.0 ** -25])
def test_small_values_beside_large_ones(q4k, ratio, qt, ct, form):   # noqa: F811
    """Rows that see only values whose scale is a small part, or none, of one beside them: at most their own size.  (A weight
    times a scale may be lost in fp16 or rounded up to its smallest number, at most to twice itself.)"""
    case, H, KH, D, page, block = dict(new=[40], len=[200], window=16), 4, 2, 64, 64, 16
    if not _takes(form, qt, qt, D, page, 1.0, 2, 0.0):
        return
    g = torch.Generator().manual_seed(12)
    ((kc, ks, keys), (vc, _, vals)), pt = _cache(g, case["len"], page, block, KH, D, ct)
    s = torch.where(torch.arange(200) < 192, ratio * 4.0, 4.0)
    vs = torch.full_like(ks, math.nan)
    at = torch.arange(0, 200, block)
    vs[pt[0].long()[at // page].cuda(), (at % page // block).cuda()] = s[at].cuda()[:, None]
    codes = vc.float().cpu()[pt[0].long()].flatten(0, 1)[:200]
    vals = [codes.double() * s.double()[:, None, None]]
    q = torch.randn(40, H, D, generator=g).to(qt)
    lse = torch.zeros(40, H, device="cuda")
    out = q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, pt.cuda(), _starts([40]), _dev([200]), window=16, lse=lse, form=form).double().cpu()
    assert q4k.device_error_flags() == 0
    _check(out.to(qt).cuda(), lse, q, keys, vals, vs, vc, case, form, page)
    mag, _, _ = plain.attention(q, keys, [v.abs() for v in vals], case, 0.125, 0.0, None, qt == F32, F16, qt)
    assert (out.abs() <= 2 * (1 + 2.0 ** -6) * mag)[:32].all()   # (2^-8 of it the output's rounding)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("qt,ct,block", [(BF16, I8, 16), (F16, E4M3, 64), (BF16, E4M3, 4), (F32, I8, 16)])
@pytest.mark.parametrize("side", [0, 1])
def test_nan_scales_that_are_seen(q4k, side, qt, ct, block, form):   # noqa: F811
    """A scale of NaN that a row sees makes that row NaN; tokens far from those that see it do not change."""
    n, length, H, KH, D, page = 600, 700, 4, 2, 64, 64
    if not _takes(form, qt, qt, D, page, 1.0, 2, 0.0):
        return
    g = torch.Generator().manual_seed(23)
    ((kc, ks, _), (vc, vs, _)), pt = _cache(g, [length], page, block, KH, D, ct)
    q = torch.randn(n, H, D, generator=g).to(qt).cuda()
    args = (pt.cuda(), _starts([n]), _dev([length]))
    want = q4k.paged_attention8(q, kc, vc, ks, vs, *args, window=40, form=form)
    p = 448   # the block that holds this position, of cache head 1
    (vs if side else ks)[int(pt[0, p // page]), p % page // block, 1] = math.nan
    lse = torch.zeros(n, H, device="cuda")
    out = q4k.paged_attention8(q, kc, vc, ks, vs, *args, window=40, lse=lse, form=form)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    rows = torch.arange(n) + length - n
    sees = (rows >= p) & (rows - 39 < p // block * block + block)
    assert torch.isnan(out[sees.cuda()][:, 2:]).all()
    assert side or torch.isnan(lse[sees.cuda()][:, 2:]).all()
    far = ((rows < p - 256) | (rows >= p + block + 40 + 256)).cuda()
    assert int(far.sum()) > 20 and torch.equal(out[far], want[far]) and torch.equal(out[:, :2], want[:, :2])
