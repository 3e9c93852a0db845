"""GPU parity of the rotary table, the rotation and the paged append against their definitions in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def q4k():
    import __graft_entry__
    __graft_entry__.build()
    import q4_dequant_gemv_gb300 as q4k
    torch.cuda.set_device(0)
    q4k.device_error_clear()
    return q4k


def _close(got, ref, bound, what):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound).max()):.3g} x the bound"


def _normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, dtype=torch.float64).to(dtype)


def _freqs(rot, base, scaling, factor, orig, low, high):
    """f_i in Python floats, from the definitions."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "ramp":
            at = lambda r: rot * math.log(orig / (2 * math.pi * r)) / (2 * math.log(base))
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
            r = min(max((i - a) / (b - a), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        elif scaling == "bands":
            wave = 2 * math.pi / f
            if wave > orig / low:
                f /= factor
            elif wave >= orig / high:
                m = (orig / wave - low) / (high - low)
                f = (1 - m) * f / factor + m * f
        out.append(f)
    return out


@pytest.mark.parametrize("rows,rot,scaling", [(1, 2, None), (1000, 128, None), (70000, 64, "linear"), (3000, 96, "base"),
                                              (40000, 128, "ramp"), (40000, 128, "bands"), (0, 64, None), (17, 512, None)])
def test_table(q4k, rows, rot, scaling):
    factor, orig = (4.0, 8192.0) if scaling else (1.0, 0.0)
    low, high = (1.0, 4.0) if scaling == "bands" else (1.0, 32.0)
    base = 500000.0 if scaling == "bands" else 10000.0
    got = q4k.rope_table(rows, rot, base, scaling=scaling, factor=factor, orig_len=orig)
    f = torch.tensor(_freqs(rot, base, scaling, factor, orig, low, high), dtype=torch.float64)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    mag = 0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0
    ref = torch.cat([a.cos(), a.sin()], 1) * mag
    # one rounding to fp32, and f_i known to a few 2^-53 of itself on an angle of `rows`
    _close(got, ref, 2.0 ** -24 * 1.25 + rows * 2.0 ** -48, "table")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("T,H,D,rot", [(1, 28, 128, 128), (3, 5, 64, 32), (17, 2, 80, 80), (9, 3, 7, 6), (2, 1, 256, 64),
                                       (33, 40, 96, 48), (5, 2, 128, 0), (4, 3, 24, 2), (2, 7, 520, 512)])
def test_rope(q4k, T, H, D, rot, xt, yt, interleaved):
    g = torch.Generator().manual_seed(T * 1000 + D)
    x = _normal(g, T, H, D, dtype=xt)
    tab = plain.table(300, rot) if rot else torch.zeros(1, 0)
    pos = torch.randint(0, 300 if rot else 1, (T,), generator=g).to(torch.int32)
    y = q4k.rope(x.cuda(), pos.cuda(), tab.cuda(), interleaved=interleaved, out_dtype=yt)
    assert y.dtype == yt and y.shape == x.shape
    ref, mag = plain.turn(x, tab[pos.long()], interleaved)
    _close(y, ref, plain.turn_bound(ref, mag, yt), "rope")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_rope_strides_in_place(q4k, dtype, pad):
    """Padded rows (pad 1 breaks the 16-byte alignment), a transposed order, and y = x."""
    g = torch.Generator().manual_seed(5 + pad)
    T, H, D, rot = 6, 4, 64, 64
    tab, pos = plain.table(50, rot), torch.arange(T, dtype=torch.int32) * 7
    buf = _normal(g, H, T, D + pad, dtype=dtype).cuda()
    x = buf.transpose(0, 1)[..., :D]
    ref, mag = plain.turn(x.cpu(), tab[pos.long()], False)
    y = torch.full((T, H, D + 2 * pad), 7.0, dtype=dtype, device="cuda")
    out = q4k.rope(x, pos.cuda(), tab.cuda(), y[..., pad:pad + D])
    _close(out, ref, plain.turn_bound(ref, mag, dtype), "strided")
    assert torch.all(y[..., :pad] == 7.0) and torch.all(y[..., pad + D:] == 7.0)
    margin = buf[..., D:].clone()
    assert q4k.rope(x, pos.cuda(), tab.cuda(), x).data_ptr() == x.data_ptr()
    _close(x, ref, plain.turn_bound(ref, mag, dtype), "in place")
    assert torch.equal(buf[..., D:], margin)


def test_rope_far_positions(q4k):
    """Positions of 100,000 and more keep fp32 accuracy through the table."""
    tab = q4k.rope_table(131072, 128)
    pos = torch.tensor([131071, 100001, 65537, 0], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    x = _normal(g, 4, 2, 128)
    f = torch.tensor([10000.0 ** (-2.0 * i / 128) for i in range(64)], dtype=torch.float64)
    a = pos.double()[:, None] * f
    ref, mag = plain.turn(x, torch.cat([a.cos(), a.sin()], 1), False)
    y = q4k.rope(x.cuda(), pos.cuda(), tab)
    # the table's own rounding on top of the arithmetic's
    _close(y, ref, plain.turn_bound(ref, mag, F32) + 2.0 ** -23 * (x.abs().amax(-1, keepdim=True).double() * 2), "far")


def test_rope_bad_position_is_not_followed(q4k):
    x = torch.ones(3, 1, 64, device="cuda")
    y = torch.full_like(x, 5.0)
    pos = torch.tensor([0, 10, -1], dtype=torch.int32, device="cuda")
    q4k.rope(x, pos, plain.table(10, 64).cuda(), y)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 4
    q4k.device_error_clear()
    assert torch.equal(y[0], x[0]) and torch.all(y[1:] == 5.0)


APPEND = [
    # new tokens, lengths, heads, kv heads, dim, rot, page, heads first
    ([1], [1], 28, 4, 128, 128, 16, False),
    ([1, 1, 1], [17, 16, 1], 8, 8, 64, 64, 16, True),
    ([5, 0, 33, 1], [5, 9, 100, 64], 14, 2, 96, 48, 48, False),
    ([7, 20], [7, 31], 3, 1, 80, 80, 5, False),
    ([300], [1000], 4, 4, 128, 64, 1, True),
    ([2, 3], [2, 50], 6, 3, 10, 6, 7, False),
    ([1] * 300, list(range(1, 301)), 2, 1, 64, 64, 32, False),
]


@pytest.mark.parametrize("types", [(F32, BF16, F32), (F32, F16, BF16), (BF16, BF16, BF16), (F16, F16, F16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,lens,H,KH,D,rot,page,first", APPEND)
def test_append(q4k, new, lens, H, KH, D, rot, page, first, types, interleaved):
    kt, ct, qo = types
    g = torch.Generator().manual_seed(sum(lens) + D)
    T, B = sum(new), len(new)
    k, v, q = (_normal(g, T, h, D, dtype=kt) for h in (KH, KH, H))
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 2
    perm = torch.randperm(pages, generator=g).tolist()
    pt = torch.full((B, max(counts)), -1, dtype=torch.int32)
    for b, c in enumerate(counts):
        for i in range(c):
            pt[b, i] = perm.pop()
    shape = (pages, KH, page, D) if first else (pages, page, KH, D)
    kc = torch.randn(*shape, generator=g).to(ct)
    vc = torch.randn(*shape, generator=g).to(ct)
    kd, vd = kc.cuda(), vc.cuda()
    view = (lambda t: t.transpose(1, 2)) if first else (lambda t: t)
    start = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32)
    ln = torch.tensor(lens, dtype=torch.int32)
    tab = plain.table(max(lens), rot)
    out = q4k.kv_append(k.cuda(), v.cuda(), view(kd), view(vd), pt.cuda(), start.cuda(), ln.cuda(), table=tab.cuda(),
                        interleaved=interleaved, q=q.cuda(), q_dtype=qo)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    where = [(b, lens[b] - new[b] + i) for b in range(B) for i in range(new[b])]
    pos = torch.tensor([p for _, p in where], dtype=torch.int64)
    ref, mag = plain.turn(q, tab[pos], interleaved)
    assert out.dtype == qo
    _close(out, ref, plain.turn_bound(ref, mag, qo), "q")
    ref, mag = plain.turn(k, tab[pos], interleaved)
    page_of = torch.tensor([int(pt[b, p // page]) for b, p in where])
    slot = pos % page
    _close(view(kd).cpu()[page_of, slot], ref, plain.turn_bound(ref, mag, ct), "k")
    assert torch.equal(view(vd).cpu()[page_of, slot], v.to(ct)), "values are rounded once"
    # nothing else of the cache changed
    for dev, host in ((kd, kc), (vd, vc)):
        a, b = view(dev.cpu()).clone(), view(host).clone()
        a[page_of, slot] = 0
        b[page_of, slot] = 0
        assert torch.equal(a, b)


def test_append_own_positions_no_table_and_in_place_q(q4k):
    g = torch.Generator().manual_seed(9)
    k, v, q = (_normal(g, 4, 2, 64).cuda() for _ in range(3))
    kc, vc = (torch.zeros(3, 16, 2, 64, dtype=BF16, device="cuda") for _ in range(2))
    pt = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ln = torch.tensor([18], dtype=torch.int32, device="cuda")
    assert q4k.kv_append(k, v, kc, vc, pt, start, ln) is None
    want = torch.zeros_like(kc)
    want[2, 14:16], want[0, 0:2] = k[:2].to(BF16), k[2:].to(BF16)
    assert torch.equal(kc, want)
    pos = torch.tensor([3, 1, 4, 1], dtype=torch.int32)
    tab = plain.table(5, 64)
    ref, mag = plain.turn(q.cpu(), tab[pos.long()], False)
    assert q4k.kv_append(k, v, kc, vc, pt, start, ln, table=tab.cuda(), pos=pos.cuda(), q=q, q_out=q) is q
    _close(q, ref, plain.turn_bound(ref, mag, F32), "q in place")
    assert q4k.device_error_flags() == 0


def test_append_bad_indices_are_not_followed(q4k):
    """A page outside the cache, a position past the page table, one before 0: skipped and flagged, the rest written."""
    k = torch.ones(4, 1, 64, device="cuda")
    tab = plain.table(4, 64).cuda()
    for pt, start, ln, ok in [([[5, 0]], [0, 4], [18], 2), ([[-1, 0]], [0, 4], [18], 2), ([[0, 1]], [0, 4], [34], 2),
                              ([[0, 1]], [0, 4], [2], 2), ([[0, 1]], [0, 9], [9], 0)]:
        kc, vc = (torch.zeros(3, 16, 1, 64, dtype=F16, device="cuda") for _ in range(2))
        dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (pt, start, ln)]
        q4k.kv_append(k, k, kc, vc, *dev)
        torch.cuda.synchronize()
        assert q4k.device_error_flags() == 4
        q4k.device_error_clear()
        assert int((vc != 0).any(-1).sum()) == ok
    kc, vc = (torch.zeros(3, 16, 1, 64, dtype=F16, device="cuda") for _ in range(2))
    dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0, 1]], [0, 4], [8])]
    q4k.kv_append(k, k, kc, vc, *dev, table=tab)     # rows 4..7 of a table of 4
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 4 and not vc.any()
    q4k.device_error_clear()


def test_refusals(q4k):
    x = torch.zeros(2, 3, 64, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    tab = plain.table(4, 64).cuda()
    kc = torch.zeros(2, 16, 3, 64, dtype=BF16, device="cuda")
    pt = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    ln = torch.tensor([2], dtype=torch.int32, device="cuda")
    ok = dict(k=x, v=x, k_cache=kc, v_cache=kc.clone(), page_table=pt, seq_start=start, kv_len=ln)
    for bad, err in [(lambda: q4k.rope(x.double(), pos, tab), TypeError), (lambda: q4k.rope(x[0], pos, tab), ValueError),
                     (lambda: q4k.rope(x, pos.long(), tab), TypeError), (lambda: q4k.rope(x, pos[:1], tab), ValueError),
                     (lambda: q4k.rope(x, pos, plain.table(4, 66).cuda()), ValueError),
                     (lambda: q4k.rope(x, pos, tab.half()), TypeError), (lambda: q4k.rope(x.cpu(), pos, tab), ValueError),
                     (lambda: q4k.rope(x, None, tab), ValueError),
                     (lambda: q4k.rope(x, pos, tab, x[:, :2]), ValueError),
                     (lambda: q4k.rope(x.transpose(1, 2), pos, tab), ValueError),
                     (lambda: q4k.rope_table(8, 3), ValueError), (lambda: q4k.rope_table(8, 8, scaling="other"), ValueError),
                     (lambda: q4k.rope_table(8, 1024), q4k.Q4KError), (lambda: q4k.rope_table(8, 8, -1.0), q4k.Q4KError),
                     (lambda: q4k.rope_table(8, 8, scaling="ramp", factor=2.0), q4k.Q4KError),
                     (lambda: q4k.kv_append(**{**ok, "v": x.half()}), TypeError),
                     (lambda: q4k.kv_append(**{**ok, "v": x[:1]}), ValueError),
                     (lambda: q4k.kv_append(**{**ok, "k_cache": kc.float()}), TypeError),
                     (lambda: q4k.kv_append(**{**ok, "k_cache": kc[:1]}), ValueError),
                     (lambda: q4k.kv_append(**{**ok, "k": x[:, :2], "v": x[:, :2]}), ValueError),
                     (lambda: q4k.kv_append(**{**ok, "kv_len": ln.long()}), TypeError),
                     (lambda: q4k.kv_append(**{**ok, "seq_start": start[:1]}), ValueError),
                     (lambda: q4k.kv_append(**{**ok, "page_table": pt[0]}), ValueError),
                     (lambda: q4k.kv_append(**ok, q_out=x), ValueError)]:
        with pytest.raises(err):
            bad()
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0 and not kc.any()
