"""Prompt chunks over 8-bit caches with blocks of 16 tokens or more: the many-rows form multiplies the codes themselves, exact
in fp16, so scores are as close as over a 16-bit cache.  The bounds here have no room for keys rounded after their scale."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402
import plain_cache8 as plain8     # noqa: E402
from test_attention8_gpu import BF16, E4M3, F16, I8, _cache, _dev, q4k   # noqa: E402,F401

pytestmark = pytest.mark.gpu


def _score_error(q, keys, case, scale):
    """What fp32 accumulation (dim 2^-23 of the terms' sizes, as in plain_attention) and scaling may cost a row's scores."""
    T, H, D = q.shape
    off = torch.zeros(T, H, dtype=torch.float64)
    for t, (b, _, lo, hi) in enumerate(plain.ranges(case)):
        k = keys[b][lo:hi].repeat_interleave(H // keys[b].shape[1], 1)
        size = torch.einsum("hd,jhd->hj", q[t].double().abs(), k.abs()) * scale
        s = torch.einsum("hd,jhd->hj", q[t].double(), k) * scale
        off[t] = (D + 8) * 2.0 ** -23 * size.amax(1) + 2.0 ** -21 * s.abs().amax(1)
    return off


@pytest.mark.parametrize("qt,ct", [(BF16, I8), (F16, I8), (BF16, E4M3), (F16, E4M3)])
@pytest.mark.parametrize("D,page,block", [(64, 64, 16), (64, 32, 32), (128, 128, 64), (128, 16, 16), (96, 128, 128)])
def test_codes_stay_exact(q4k, D, page, block, qt, ct):   # noqa: F811
    case, H, KH, scale = dict(new=[40, 130], len=[300, 140]), 6, 2, 1.0 / math.sqrt(D)
    g = torch.Generator().manual_seed(D + block)
    ((kc, ks, keys), (vc, vs, vals)), pt = _cache(g, case["len"], page, block, KH, D, ct, spread=0.5)
    q = (torch.randn(170, H, D, generator=g) * 8).to(qt)
    lse = torch.zeros(170, H, device="cuda")
    out = q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, pt.cuda(), _dev([0, 40, 170]), _dev(case["len"]), lse=lse, form="many")
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    ref, rl, bound = plain.attention(q, keys, vals, case, scale, parts=False, cache_dtype=F16, out_dtype=qt)
    # A weight's exponent takes three roundings beside its score's (the factor's logarithm, its difference from the maximum, the
    # sum), each 2^-24 of a number below |lse| / ln 2 + 2^5: 2^-22 |lse| + 2^-18 of the weight, twice that of a quotient.  Weights of
    # 2^6 at least over 2^t, at most twice the largest scale, lose 2^-25 in fp16: 2^-30 of that scale.
    few = float(vs[torch.isfinite(vs)].max()) * 2.0 ** -30 * plain8.TOP[ct] * max(case["len"])
    mag, _, _ = plain.attention(q, keys, [v.abs() for v in vals], case, scale, parts=False, cache_dtype=F16, out_dtype=qt)
    assert ((out.double().cpu() - ref).abs() <= bound + (2.0 ** -21 * rl.abs() + 2.0 ** -17)[..., None] * mag + few).all()
    # the log-sum-exp: the scores' error, the exponents', its own rounding
    tol = _score_error(q, keys, case, scale) + 2.0 ** -17 + 2.0 ** -22 * rl.abs()
    assert ((lse.double().cpu() - rl).abs() <= tol).all()
    # keys rounded to fp16 after their scale would not pass
    rounded = [(k / 2.0 ** -6).to(F16).double() * 2.0 ** -6 for k in keys]
    _, wrong, _ = plain.attention(q, rounded, vals, case, scale, parts=False, cache_dtype=F16, out_dtype=qt)
    assert ((wrong - rl).abs() > tol).double().mean() > 0.2
