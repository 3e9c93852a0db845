"""Document masks that leave holes: tokens that see nothing between tokens that do (padding), whose slots nobody sees.
Keys and values there are NaN or infinite, whole pages there are missing from the page table; all forms of the kernels."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402
from test_attention_forms_gpu import FORMS, _takes   # noqa: E402
from test_attention_gpu import BF16, F16, F32, _dev, q4k   # noqa: E402,F401

pytestmark = pytest.mark.gpu
NOTHING = 10 ** 9


def _padded(n, length, seen, first=0):
    """kv_start of n new tokens: `seen` holds the ranges of new tokens (in order) that see the keys from `first` on
    (the first range) or from their range's start on; the tokens between see nothing."""
    out, past = [NOTHING] * n, length - n
    for k, (a, b) in enumerate(seen):
        for i in range(a, b):
            out[i] = first if k == 0 else past + a
    return out


CASES = [
    dict(new=[3], len=[13], kv_start=_padded(3, 13, [(0, 1), (2, 3)])),
    dict(new=[3, 5], len=[13, 70], kv_start=_padded(3, 13, [(1, 2)]) + _padded(5, 70, [(0, 2), (4, 5)])),
    dict(new=[120], len=[300], kv_start=_padded(120, 300, [(0, 40), (80, 120)])),
    dict(new=[200, 1, 64], len=[900, 20, 64],
         kv_start=_padded(200, 900, [(0, 1), (60, 61), (150, 200)], 400) + [0] + _padded(64, 64, [(0, 3), (50, 64)])),
    dict(new=[100], len=[400], prefix=[50], kv_start=_padded(100, 400, [(0, 1), (49, 50), (90, 100)])),
    dict(new=[90], len=[333], window=25, kv_start=_padded(90, 333, [(0, 20), (60, 90)])),
    # tiles that see nothing at all
    dict(new=[1, 2], len=[18, 100], causal=False, kv_start=[NOTHING, 100, NOTHING]),
    dict(new=[40, 300], len=[57, 700], causal=False, kv_start=[NOTHING] * 40 + [650] * 20 + [700] * 280),
    dict(new=[1, 40], len=[18, 77], kv_start=[18] + [NOTHING] * 40),
]


@pytest.mark.parametrize("form", [None, *FORMS])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
@pytest.mark.parametrize("H,KH,D,page,types,fill", [
    (4, 4, 64, 16, (BF16, BF16, BF16), math.nan), (14, 2, 128, 64, (F16, F16, F16), math.inf),
    (8, 2, 64, 32, (F32, BF16, F32), math.nan), (4, 1, 128, 5, (F32, F16, F32), math.inf),
    (2, 2, 192, 16, (BF16, BF16, BF16), math.nan)])
def test_holes(q4k, case, H, KH, D, page, types, fill, form):   # noqa: F811
    qt, ct, ot = types
    g = torch.Generator().manual_seed(17 + H + D + len(case["kv_start"]))
    seen = [torch.zeros(n, dtype=torch.bool) for n in case["len"]]
    for b, _, lo, hi in plain.ranges(case):
        seen[b][lo:hi] = True
    q = (torch.randn(sum(case["new"]), H, D, generator=g, dtype=torch.float64) * 1.5).to(qt)
    keys, vals = ([torch.randn(n, KH, D, generator=g).to(ct) for n in case["len"]] for _ in range(2))
    order = torch.randperm(sum(-(-n // page) for n in case["len"]) + 2, generator=g)
    for k, v, s in zip(keys, vals, seen):
        k[~s], v[~s] = fill, -fill
    kc, pt = plain.paged(keys, page, ct, order, fill=fill)
    vc, _ = plain.paged(vals, page, ct, order, fill=-fill)
    for b, s in enumerate(seen):
        for i in range(-(-s.numel() // page)):
            if not s[i * page:(i + 1) * page].any():
                pt[b, i] = -1
    kc, vc = kc.cuda(), vc.cuda()
    if form and not _takes(form, q, kc, ot, None):
        pytest.skip("the form does not take the call")
    start = _dev([sum(case["new"][:i]) for i in range(len(case["new"]) + 1)])
    lse = torch.zeros(q.shape[0], H, device="cuda")
    out = q4k.paged_attention(q.cuda(), kc, vc, pt.cuda(), start, _dev(case["len"]), out_dtype=ot, lse=lse, form=form,
                              causal=case.get("causal", True), window=case.get("window", 0), prefix_len=_dev(case.get("prefix")), kv_start=_dev(case["kv_start"]))
    torch.cuda.synchronize()
    flags = q4k.device_error_flags()
    q4k.device_error_clear()
    assert flags == 0
    ref, rl, bound = plain.attention(q, keys, vals, case, 1.0 / math.sqrt(D), parts=qt != ct or ot == F32, cache_dtype=ct,
                                     out_dtype=ot)
    assert ((out.double().cpu() - ref).abs() <= bound).all()
    assert not out.cpu()[torch.isinf(rl)].any() and torch.equal(torch.isinf(rl), torch.isinf(lse.cpu()))
