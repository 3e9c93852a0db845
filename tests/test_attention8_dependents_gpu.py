"""Append and the many-rows form over an 8-bit cache as programmatic dependents of each other, over and over into the same
slots: each call reads what the one before it wrote."""
import pytest

torch = pytest.importorskip("torch")
from test_attention8_gpu import BF16, E4M3, F16, I8, _dev, q4k   # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qt,ct,block", [(BF16, I8, 16), (F16, E4M3, 1), (BF16, E4M3, 64)])
def test_dependents_over_the_same_slots(q4k, qt, ct, block):   # noqa: F811
    n, H, KH, D, page, steps = 300, 8, 4, 128, 64, 12
    g = torch.Generator(device="cuda").manual_seed(41)
    pt = torch.randperm(12, generator=g, device="cuda").to(torch.int32).view(2, 6)
    start, ln = _dev([0, n, 2 * n]), _dev([n + 30, n])
    data = [[torch.randn(2 * n, h, D, generator=g, device="cuda").to(qt) for h in (KH, KH, H)] for _ in range(steps)]
    table = q4k.rope_table(400, D)

    def run(pdl):
        cache = [torch.zeros(12, page, KH, D, dtype=torch.uint8, device="cuda").view(ct) for _ in range(2)] + \
            [torch.zeros(12, page // block, KH, device="cuda") for _ in range(2)]
        outs = []
        for k, v, q in data:
            a = q4k.kv_append8(k, v, *cache, pt, start, ln, table=table, q=q, pdl=pdl)
            outs.append(q4k.paged_attention8(a, *cache, pt, start, ln, form="many", pdl=pdl))
            if not pdl:
                torch.cuda.synchronize()
        return outs

    want = run(False)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(run(True), want))
    assert q4k.device_error_flags() == 0
