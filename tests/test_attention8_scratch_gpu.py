"""What the widened form over an 8-bit cache leaves with the library: a page table far wider than its sequences asks for
gigabytes of scratch, which go back to the system."""
import pytest

torch = pytest.importorskip("torch")
from test_attention8_gpu import I8, _cache, _dev, q4k   # noqa: E402,F401

pytestmark = pytest.mark.gpu
GIB = 2 ** 30


@pytest.mark.parametrize("keep", [GIB, 0])
def test_scratch_goes_back(q4k, keep):   # noqa: F811
    """A call over a table of 4 GiB of widened keys and values: once the program has synchronised, what it was told is kept at
    most; the results are the same."""
    g = torch.Generator().manual_seed(3)
    KH, D, page, lens = 2, 128, 64, [300, 140]
    ((kc, ks, _), (vc, vs, _)), pt = _cache(g, lens, page, 16, KH, D, I8)
    wide = torch.full((2, (4 * GIB // (2 * KH * 4 * D) - 4096) // page), -1, dtype=torch.int32)
    wide[:, :pt.shape[1]] = pt
    q = torch.randn(200, 4, D, generator=g).bfloat16().cuda()
    args = (q, kc, vc, ks, vs, wide.cuda(), _dev([0, 100, 200]), _dev(lens))
    want = q4k.paged_attention8(*args, form="many")
    q4k.scratch_keep(keep)
    try:
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        outs = [q4k.paged_attention8(*args, form="many") for _ in range(3)]
        during = before - torch.cuda.mem_get_info()[0]
        for _ in range(2):
            torch.cuda.synchronize()
        lost = before - torch.cuda.mem_get_info()[0]
        assert during > 2.5 * GIB and lost < keep + GIB // 4, f"{during / GIB:.2f} GiB taken, {lost / GIB:.2f} kept"
        assert all(torch.equal(x, want) for x in outs)
    finally:
        q4k.scratch_keep(5 * GIB)
    assert torch.equal(q4k.paged_attention8(*args, form="many"), want)
    assert q4k.device_error_flags() == 0
