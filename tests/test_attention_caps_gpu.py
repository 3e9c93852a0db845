"""Caps on the scores far from the usual 30 to 50: a large one leaves the scores as they are, a tiny one makes them equal."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402
from test_attention_gpu import BF16, F16, F32, _dev, q4k   # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [1e-40, 1e-3, 200.0, 1e3, 1e5, 1e8, 1e20, 3e38])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F16, F16, F16), (F32, BF16, F32), (F32, F16, F32)])
@pytest.mark.parametrize("new,lens", [([1], [700]), ([3, 1], [50, 90]), ([200], [500])])
def test_caps(q4k, new, lens, types, cap):   # noqa: F811
    """Against the definition in 64 bits.  The bound: that of uncapped scores (the cap's slope is at most 1), and the
    cap's own: 2^-20 of a score where it is formed with relative precision, 2^-21 of the cap up to 256 otherwise
    (there the sum 1 - 2 / (exp + 1) is off by 2^-22)."""
    qt, ct, ot = types
    H, KH, D, page = 8, 2, 64, 16
    g = torch.Generator().manual_seed(int(math.log2(cap)) + 400 + sum(lens))
    case = dict(new=new, len=lens)
    q = (torch.randn(sum(new), H, D, generator=g, dtype=torch.float64) * 2.0).to(qt)
    keys, vals = ([torch.randn(n, KH, D, generator=g).to(ct) for n in lens] for _ in range(2))
    order = torch.randperm(sum(-(-n // page) for n in lens) + 2, generator=g)
    kc, pt = plain.paged(keys, page, ct, order)
    vc, _ = plain.paged(vals, page, ct, order)
    start = _dev([sum(new[:i]) for i in range(len(new) + 1)])
    out = q4k.paged_attention(q.cuda(), kc.cuda(), vc.cuda(), pt.cuda(), start, _dev(lens), out_dtype=ot, softcap=cap)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    scale = 1.0 / math.sqrt(D)
    many = qt != ct or ot == F32
    ref, _, _ = plain.attention(q, keys, vals, case, scale, cap, None, many, ct, ot)
    _, _, bound = plain.attention(q, keys, vals, case, scale, 0.0, None, many, ct, ot)
    largest = max(float(torch.einsum("thd,jhd->thj", q.double()[:, ::H // KH], k.double()).abs().max()) for k in keys) * scale * 2
    own = min(cap, largest) * 2.0 ** -20 + (cap * 2.0 ** -21 if cap <= 256 else 0.0)
    size = max(float(v.double().abs().max()) for v in vals)
    # (with equal scores the weights, and so the sums' errors, spread over all keys)
    flat = (16 + math.sqrt(max(lens))) * 2.0 ** -21 * size + plain.UNIT[ot] * ref.abs() + (0 if many else plain.UNIT[ct] * size)
    assert ((out.double().cpu() - ref).abs() <= bound + 2 * own * size + flat).all()
