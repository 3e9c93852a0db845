"""GPU parity of attention over an 8-bit paged cache against its definition in 64 bits: code types, blocks, head layouts,
lengths, page sizes, masks, over every form of the kernels.  Slots that hold no position have codes of NaN (e4m3) or -128,
blocks that hold none a scale of NaN, and unused page table entries are -1."""
import math
import time

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402
import plain_cache8 as plain8     # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn
FORMS = [None, "cluster8", "cluster16", "cluster32", "split8", "split16", "split32", "many"]


@pytest.fixture(scope="module")
def q4k():
    import __graft_entry__
    __graft_entry__.build()
    import q4_dequant_gemv_gb300 as q4k
    torch.cuda.set_device(0)
    q4k.device_error_clear()
    return q4k


def _dev(x):
    return None if x is None else torch.as_tensor(x, dtype=torch.int32).cuda()


def _bytes(t):
    return t.view(torch.uint8)


def _cache(g, lens, page, block, KH, D, ct, first=False, spare=2, spread=1.0):
    """[(codes, scales) of keys and values] on the device, the page table, and the values [len, KH, D] in 64 bits."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=g)
    pt = torch.full((len(lens), max(counts + [1])), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        pt[b, :c] = order[at:at + c]
        at += c
    sides = []
    for _ in range(2):
        codes = torch.full((pages, page, KH, D), 0x7F if ct == E4M3 else 0x80, dtype=torch.uint8)
        scales = torch.full((pages, page // block, KH), float("nan"))
        vals = []
        for b, n in enumerate(lens):
            x = torch.randn(n, KH, D, generator=g)
            blocks = torch.arange(n) // block
            s = torch.exp(torch.randn(n // block + 1, KH, generator=g) * spread)[blocks] * 0.03
            if ct == I8:
                c = (x * 32).round().clamp(-127, 127).to(I8)
            else:
                c = (x * 32).to(E4M3)
            page_of, slot = pt[b].long()[torch.arange(n) // page], torch.arange(n) % page
            codes[page_of, slot] = _bytes(c)
            scales[page_of, slot // block] = s
            vals.append(c.float().double() * s.double()[..., None])
        codes = codes.cuda()
        codes = codes.transpose(1, 2).contiguous().transpose(1, 2) if first else codes
        sides.append((codes.view(ct), scales.cuda(), vals))
    return sides, pt


def _floor(vs, vc, lens, many=False):
    """Softmax weights go to fp16 as e s 2^(14 - t), e the weight over the largest, s the value's scale, 2^t at most twice the
    largest scale: below fp16's normal numbers each (and the last part of one in parts) is off by half a step, 2^-25, so
    e s by 2^-39 2^t <= 2^-38 max s, and an output by that times the codes it sums, over a sum of weights of at least 1.
    (It shows where the keys of large weight have codes of 0.)  The many-rows form has e 2^6 f / 2^t, f the factor of a piece of
    values, 2^t at most twice the largest, and rows of up to 128 times their codes: 2^-25 2^-6 2^t 128 / 64 <= 2^-29 max s."""
    s = vs[torch.isfinite(vs)]
    return 2.0 ** (-29 if many else -38) * (float(s.max()) if s.numel() else 0.0) * plain8.TOP[vc.dtype] * max(lens)


def _products(q, keys, vals, case, scale, slopes, softcap):
    """What the many-rows form adds to the bound: keys and values over their units' powers of two are rounded to fp16, the
    products with a key's scale once (2^-11 of itself), with a value's twice (its scale too), so a score is off by at most
    2^-11 of its terms' sizes, as much as that the log-sum-exp (returned beside it), and a weight by twice that."""
    T, H, D = q.shape
    out, off = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t, (b, p, lo, hi) in enumerate(plain.ranges(case)):
        if hi <= lo:
            continue
        g = H // keys[b].shape[1]
        k, v = (x[b][lo:hi].repeat_interleave(g, 1) for x in (keys, vals))
        s = torch.einsum("hd,jhd->hj", q[t].double(), k) * scale
        size = torch.einsum("hd,jhd->hj", q[t].double().abs(), k.abs()) * abs(scale)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes.double()[:, None] * (p - torch.arange(lo, hi, dtype=torch.float64)).abs()
        mag = torch.einsum("hj,jhd->hd", torch.softmax(s, 1), v.abs())
        off[t] = 2.0 ** -11 * size.amax(1)
        out[t] = (2 * off[t][:, None] + 2 * 2.0 ** -11) * mag
    return out, off


def _takes(form, qt, ot, D, page, scale, group, cap):
    if form == "many":
        return qt != F32 and ot != F32 and D <= 128 and page % 16 == 0 and scale >= 0 and group <= 256 and cap <= 256
    return form is None or D <= 128 or not form.endswith("32")


def _run(q4k, case, H, KH, D, page, block=16, qt=BF16, ct=I8, ot=None, softcap=0.0, slopes=None, first=False, scale=None,
         std=1.5, seed=0, form=None, spread=1.0):
    """Builds the call, checks out and lse; returns (out, the call), or None where the form is refused."""
    ot = qt if ot is None else ot
    g = torch.Generator().manual_seed(seed * 7919 + sum(case["len"]) * 31 + H * D)
    T = sum(case["new"])
    q = (torch.randn(T, H, D, generator=g, dtype=torch.float64) * std).to(qt)
    (kc, ks, keys), (vc, vs, vals) = (sides := _cache(g, case["len"], page, block, KH, D, ct, first, spread=spread))[0]
    pt = sides[1]
    if case.get("window") and case.get("free"):     # pages that no window reaches any more
        for b, (n, length) in enumerate(zip(case["new"], case["len"])):
            pt[b, :max(0, length - n + 1 - case["window"]) // page] = -1
    start = _dev([sum(case["new"][:i]) for i in range(len(case["new"]) + 1)])
    lse = torch.full((T, H), 7.0, device="cuda")
    sl = None if slopes is None else torch.tensor(slopes, dtype=F32)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    args = (q.cuda(), kc, vc, ks, vs, pt.cuda(), start, _dev(case["len"]))
    kw = dict(scale=scale, out_dtype=ot, softcap=softcap, slopes=None if sl is None else sl.cuda(),
              window=case.get("window", 0), causal=case.get("causal", True), prefix_len=_dev(case.get("prefix")),
              kv_start=_dev(case.get("kv_start")), form=form)
    if not _takes(form, qt, ot, D, page, scale, H // KH, softcap):
        with pytest.raises(q4k.Q4KError) as e:
            q4k.paged_attention8(*args, **kw)
        assert e.value.status == 1
        return None
    out = q4k.paged_attention8(*args, lse=lse, **kw)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    assert out.dtype == ot and tuple(out.shape) == (T, H, D)
    # the same sums as over a cache of fp16: weights rounded once to fp16, or both in parts of 22 bits
    many = qt == F32 or ot == F32 or softcap > 256
    ref, rl, bound = plain.attention(q, keys, vals, case, scale, softcap, sl, many, F16, ot)
    chunk = not many and D <= 128 and page % 16 == 0 and form in (None, "many")   # (or may be)
    bound = bound + _floor(vs, vc, case["len"], chunk) + (more := _products(q, keys, vals, case, scale, sl, softcap) if chunk else (0.0, 0.0))[0]
    err = (out.double().cpu() - ref).abs()
    assert (err <= bound).all(), f"out: worst {float((err / bound).max()):.3g} x the bound"
    dead = torch.isinf(rl)
    got = lse.double().cpu()
    assert torch.equal(dead, torch.isinf(got) & (got < 0))
    assert not out.cpu()[dead].any(), "a row that sees nothing is zero"
    # the scores' own errors (bounded well inside 2^-12 here) and fp32's on the sum
    tol = 2.0 ** -12 + 2.0 ** -20 * rl[~dead].abs() + (more[1][~dead] if chunk else 0.0)
    assert ((got[~dead] - rl[~dead]).abs() <= tol).all()
    return out, lambda **over: q4k.paged_attention8(*args, **{**kw, **over})


TYPES = [(BF16, I8, BF16), (F16, E4M3, F16), (F32, I8, F32), (F32, E4M3, F32), (BF16, E4M3, F32), (F16, I8, BF16)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new,lens,H,KH,D,page,block", [
    ([1], [1], 28, 4, 128, 16, 16),
    ([1, 1, 1], [300, 17, 128], 28, 4, 128, 16, 1),
    ([5, 5], [40, 261], 28, 4, 128, 64, 4),
    ([1, 0, 40, 3], [9, 12, 200, 3], 8, 8, 64, 32, 32),
    ([70], [333], 6, 2, 128, 64, 64),
])
def test_types(q4k, new, lens, H, KH, D, page, block, types, form):
    _run(q4k, dict(new=new, len=lens), H, KH, D, page, block, *types, form=form)


@pytest.mark.parametrize("H,KH,D", [(4, 4, 16), (8, 1, 64), (32, 1, 128), (9, 3, 80), (5, 5, 96), (16, 2, 112), (3, 1, 48),
                                    (7, 1, 144), (4, 2, 192), (16, 4, 256), (40, 1, 64)])
@pytest.mark.parametrize("form", FORMS)
def test_heads_and_dims(q4k, H, KH, D, form):
    case = dict(new=[1, 4, 37], len=[200, 65, 131])
    for types in ((BF16, I8, BF16), (F32, E4M3, F32)):
        _run(q4k, case, H, KH, D, 16, 4, *types, form=form)


@pytest.mark.parametrize("page,block", [(1, 1), (3, 1), (8, 8), (16, 2), (24, 8), (48, 16), (64, 64), (100, 4), (128, 128), (256, 32)])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("types", [(BF16, I8, BF16), (F32, E4M3, F32)])
def test_page_sizes(q4k, page, block, first, types):
    for D in (128, 64):
        for form in (None, "many"):
            _run(q4k, dict(new=[1, 150, 2], len=[513, 277, 2]), 14, 2, D, page, block, *types, first=first, form=form)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("past", [0, 1, 100])
def test_lengths(q4k, n, past):
    for form in (None, "many"):
        _run(q4k, dict(new=[n], len=[n + past]), 4, 2, 64, 16, 1, seed=n, form=form)


MASKS = [
    dict(window=1), dict(window=16), dict(window=100, free=True), dict(causal=False), dict(causal=False, window=30),
    dict(prefix=[50, 0, 1000, 3]), dict(prefix=[5, 300, 0, 0], window=20),
    dict(kv_start="docs"), dict(kv_start="docs", prefix=[10, 40, 0, 200]), dict(kv_start="beyond"), dict(kv_start="late"),
    dict(kv_start="docs", causal=False, window=7),
]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("H,KH,D,page,block,types", [(4, 2, 128, 16, 1, (BF16, E4M3, BF16)), (14, 2, 64, 32, 8, (F16, I8, F16)),
                                                     (7, 1, 96, 5, 1, (F32, E4M3, F32))])
def test_masks(q4k, mask, H, KH, D, page, block, types, form):
    case = dict(new=[90, 1, 20, 3], len=[300, 130, 20, 260], **mask)
    if mask.get("kv_start"):
        starts = []
        for n, length in zip(case["new"], case["len"]):
            for i in range(n):
                p = length - n + i
                if mask["kv_start"] == "docs":
                    starts.append(p // 37 * 37)
                elif mask["kv_start"] == "late":   # tokens that see nothing before tokens that start after them: holes
                    starts.append(p + 1 if i % 7 == 3 else max(0, p - 2))
                else:       # every third token sees nothing, one far past the end, one negative
                    starts.append(10 ** 9 if i % 3 == 0 else (-5 if i % 3 == 1 else p))
        case["kv_start"] = starts
    _run(q4k, case, H, KH, D, page, block, *types, form=form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("types", [(BF16, I8, BF16), (F32, E4M3, F32)])
@pytest.mark.parametrize("softcap,biased,causal", [(30.0, False, True), (0.0, True, True), (50.0, True, True), (5.0, True, False),
                                                   (1000.0, False, True)])
def test_cap_and_bias(q4k, types, softcap, biased, causal, form):
    H = 8
    slopes = [2.0 ** (-i - 1) for i in range(H)] if biased else None
    _run(q4k, dict(new=[1, 100, 6], len=[400, 150, 70], causal=causal), H, 4, 128, 16, 16, *types, softcap=softcap,
         slopes=slopes, std=4.0, form=form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("types", [(BF16, I8, BF16), (F32, E4M3, F32)])
@pytest.mark.parametrize("new,lens", [([1], [20000]), ([3, 1], [5000, 9001]), ([130], [6000])])
def test_long(q4k, new, lens, types, form):
    """Rows split over many CTAs."""
    _run(q4k, dict(new=new, len=lens), 8, 2, 128, 64, 16, *types, form=form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("new,lens", [([1] * 40, [70 + 13 * i for i in range(40)]), ([600], [600]), ([7, 300, 0, 64], [1500, 300, 80, 900])])
def test_many_tiles(q4k, new, lens, form):
    """More tiles than fit at once."""
    for types in ((BF16, E4M3, BF16), (F32, I8, F32)):
        _run(q4k, dict(new=new, len=lens), 14, 2, 64, 16, 4, *types, form=form)


@pytest.mark.parametrize("std", [1e-3, 40.0])
@pytest.mark.parametrize("types", [(F32, I8, F32), (BF16, E4M3, BF16)])
def test_flat_and_peaked_scores(q4k, std, types):
    for form in (None, "many"):
        _run(q4k, dict(new=[1, 33], len=[150, 260]), 4, 2, 128, 16, 16, *types, std=std, form=form)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.7])
@pytest.mark.parametrize("types", [(BF16, I8, BF16), (F32, E4M3, F32)])
def test_scales(q4k, scale, types):
    """Negative, zero and large scales of the scores, masked rows among them."""
    for new, lens in (([1], [70]), ([90, 3], [200, 40])):
        for form in (None, "many"):
            _run(q4k, dict(new=new, len=lens, window=33), 4, 2, 64, 16, 16, *types, scale=scale, form=form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("H", [130, 260])
def test_large_groups(q4k, H, form):
    """More query heads per cache head than half a tile of rows holds, and than a whole one."""
    _run(q4k, dict(new=[3, 1], len=[90, 20]), H, 1, 64, 16, 2, form=form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e-6, 1e6, 1e30])
def test_sizes_of_values(q4k, size, form):
    """Values' scales far from 1, growing and falling along the sequence, one of them zero; keys' in proportion to q."""
    n, lens, H, KH, D, page, block = 37, 400, 4, 2, 128, 16, 4
    for qt, ct in ((F32, I8), (BF16, E4M3)):
        if not _takes(form, qt, qt, D, page, 0.1, 2, 0.0):
            continue
        g = torch.Generator().manual_seed(3)
        ((kc, ks, keys), (vc, vs, _)), pt = _cache(g, [lens], page, block, KH, D, ct, spread=0.1)
        codes = vc[pt[0].long().cuda()].flatten(0, 1)[:lens].float().cpu()
        per = (torch.arange(lens) // block).double()
        s = (size * torch.exp2(per % 13 - 6)).float()
        s[(per == 20)] = 0.0
        s[per > 60] *= 64
        at = torch.arange(0, lens, block)
        vs = torch.full_like(vs, float("nan"))
        vs[pt[0].long()[at // page].cuda(), (at % page // block).cuda()] = s[at].cuda()[:, None]
        vals = [codes.double() * s.double()[:, None, None]]
        q = torch.randn(n, H, D, generator=g).to(qt)
        case = dict(new=[n], len=[lens])
        ref, _, bound = plain.attention(q, keys, vals, case, 0.1, 0.0, None, qt == F32, F16, qt)
        out = q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, pt.cuda(), _dev([0, n]), _dev([lens]), scale=0.1, form=form)
        # fp32's smallest numbers: a value's term below 2^-126 may be lost, at most one for each key and part
        err = (out.double().cpu() - ref).abs()
        many = qt != F32
        extra = _products(q, keys, vals, case, 0.1, None, 0.0)[0] if many else 0.0
        assert (err <= bound + extra + _floor(vs, vc, [lens], many) + lens * 2.0 ** -126).all(), f"{float((err / bound).max())} x the bound"
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
def test_unseen_slots_change_nothing(q4k, form):
    """Codes and scales of slots behind the sequence, before a window and of other sequences, whatever they hold."""
    new, lens, H, KH, D, page, block = [3, 40], [70, 300], 4, 2, 128, 32, 4
    for qt, ct in ((BF16, E4M3), (F32, I8)):
        if not _takes(form, qt, qt, D, page, 1.0, 2, 0.0):
            continue
        g = torch.Generator().manual_seed(5)
        ((kc, ks, _), (vc, vs, _)), pt = _cache(g, lens, page, block, KH, D, ct)
        q = torch.randn(43, H, D, generator=g).to(qt).cuda()
        args = (pt.cuda(), _dev([0, 3, 43]), _dev(lens))
        want = q4k.paged_attention8(q, kc, vc, ks, vs, *args, window=24, form=form)
        # positions that no window reaches: before len - new - 23
        for b, (n, length) in enumerate(zip(new, lens)):
            unseen = torch.arange(0, max(0, length - n - 23))
            pages, slots = pt[b].long()[unseen // page].cuda(), (unseen % page).cuda()
            for c in (kc, vc):
                _bytes(c)[pages, slots] = 0xFF if ct == E4M3 else 0x81
            whole = unseen[: len(unseen) // block * block]
            for i, s in enumerate((ks, vs)):
                s[pt[b].long()[whole // page].cuda(), (whole % page // block).cuda()] = float("inf") if i else float("nan")
        out = q4k.paged_attention8(q, kc, vc, ks, vs, *args, window=24, form=form)
        assert torch.isfinite(out).all() and torch.equal(out, want)
    assert q4k.device_error_flags() == 0


def test_nan_codes_that_are_seen(q4k):
    """An e4m3 key of NaN makes the rows that see it NaN, and no others."""
    n, lens = 15, 20
    g = torch.Generator().manual_seed(6)
    ((kc, ks, _), (vc, vs, _)), pt = _cache(g, [lens], 16, 1, 1, 64, E4M3)
    for qt, forms in ((F32, (None,)), (BF16, (None, "many"))):
        q = torch.randn(n, 1, 64, generator=g).to(qt).cuda()
        args = (pt.cuda(), _dev([0, n]), _dev([lens]))
        for form in forms:
            want = q4k.paged_attention8(q, kc, vc, ks, vs, *args, form=form)
            kn = kc.clone()
            _bytes(kn)[pt[0, 1].long(), 3] = 0x7F
            out = q4k.paged_attention8(q, kn, vc, ks, vs, *args, form=form)
            assert torch.isnan(out[-1]).all() and torch.equal(out[:-1], want[:-1])
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("n,qt", [(1, F32), (40, BF16)])
def test_strides_streams_and_graphs(q4k, n, qt):
    """Padded and transposed q and out, keys, values and scales in one buffer each, a side stream, a graph that follows the
    lengths on the device; the same bits each time."""
    g = torch.Generator().manual_seed(11)
    H, KH, D, page = 8, 2, 64, 16
    q = torch.randn(2 * n, H, D, generator=g).to(qt).cuda()
    both = torch.randint(-127, 128, (12, 2, page, KH, D), generator=g).to(I8).cuda()
    scales = torch.rand(12, 4, 2, KH, generator=g).cuda() * 0.05
    pt = torch.tensor([[3, 0, 5, 6, 7], [1, 4, 2, 8, 9]], dtype=torch.int32, device="cuda")
    start, ln = _dev([0, n, 2 * n]), _dev([70, 63])
    cache = (both[:, 0], both[:, 1], scales[:, :, 0], scales[:, :, 1])
    call = q4k.paged_attention8
    want = call(q, *(t.contiguous() for t in cache), pt, start, ln)
    wide = torch.full((H, 2 * n, D + 16), 3.0, dtype=qt, device="cuda")
    out = wide[..., :D].transpose(0, 1)
    qs = torch.zeros(H, 2 * n, D + 8, dtype=qt, device="cuda")[..., :D].transpose(0, 1)
    qs.copy_(q)
    assert call(qs, *cache, pt, start, ln, out) is out
    assert torch.equal(out, want) and torch.all(wide[..., D:] == 3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = call(q, *cache, pt, start, ln, stream=side)
    side.synchronize()
    assert torch.equal(o2, want)
    graph, o3 = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        call(q, *cache, pt, start, ln, o3)
    for _ in range(3):
        o3.zero_()
        graph.replay()
        assert torch.equal(o3, want)
    ln.copy_(_dev([60, 80]))
    graph.replay()
    assert torch.equal(o3, call(q, *cache, pt, start, ln))
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("n,qt", [(1, F32), (40, BF16)])
def test_offsets_past_32_bits(q4k, n, qt):
    """Pages more than 2^32 bytes into the cache."""
    KH, D, page = 2, 64, 16
    pages = 2 ** 32 // (KH * D * page) + 40
    kc = torch.empty(pages, page, KH, D, dtype=I8, device="cuda")
    vc = torch.empty_like(kc)
    ks, vs = (torch.full((pages, 1, KH), 0.02, device="cuda") for _ in range(2))
    pt = torch.tensor([[pages - 1, 0, pages - 5, 3, pages - 2]], dtype=torch.int32)
    length = 70
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randint(-127, 128, (length, KH, D), generator=g).to(I8) for _ in range(2))
    for i, p in enumerate(pt[0].tolist()):
        part = slice(16 * i, min(length, 16 * i + 16))
        kc[p, :k[part].shape[0]] = k[part].cuda()
        vc[p, :v[part].shape[0]] = v[part].cuda()
    q = torch.randn(n, 4, D, generator=g).to(qt)
    step = float(torch.tensor(0.02))
    ref, _, bound = plain.attention(q, [k.double() * step], [v.double() * step], dict(new=[n], len=[length]), 0.125,
                                    parts=qt == F32, cache_dtype=F16, out_dtype=qt)
    for form in (None, "many") if qt == BF16 else (None,):
        out = q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, pt.cuda(), _dev([0, n]), _dev([length]), form=form)
        k8, v8 = [k.double() * step], [v.double() * step]
        extra = _products(q, k8, v8, dict(new=[n], len=[length]), 0.125, None, 0.0)[0] + 2.0 ** -29 * step * 127 * length
        assert ((out.double().cpu() - ref).abs() <= bound + (extra if qt == BF16 else 2.0 ** -38 * step * 127 * length)).all()
    k2, v2 = q4k.kv_read8(kc, vc, ks, vs, pt.cuda(), _dev([0, length]), _dev([length]), length, dtype=F32)
    assert torch.equal(k2.cpu(), k.float() * step) and torch.equal(v2.cpu(), v.float() * step)
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
def test_bad_indices_are_not_followed(q4k, form):
    """Pages outside the cache, lengths past the page table, rows outside the call: flagged, nothing followed."""
    q = torch.ones(4, 2, 64, dtype=BF16, device="cuda")
    kc = torch.ones(3, 16, 1, 64, dtype=I8, device="cuda")
    ks = torch.ones(3, 2, 1, device="cuda")
    for pt, start, ln in [([[7, 0]], [0, 4], [20]), ([[-1, 0]], [0, 4], [20]), ([[0, 1]], [0, 4], [33]),
                          ([[0, 1]], [0, 9], [20]), ([[0, 1]], [-3, 4], [20]), ([[0, 1], [1, 2]], [0, 4, 2], [20, 20]),
                          ([[0, 1]], [0, 4], [-7])]:
        for x in (q, q.float()) if form != "many" else (q,):
            q4k.paged_attention8(x, kc, kc, ks, ks, _dev(pt), _dev(start), _dev(ln), form=form)
            torch.cuda.synchronize()
            assert q4k.device_error_flags() == 4, (pt, start, ln)
            q4k.device_error_clear()


def test_nothing_to_do(q4k):
    """No tokens, no sequences, rows of no sequence, nothing cached."""
    kc, ks = torch.ones(3, 16, 1, 64, dtype=I8, device="cuda"), torch.ones(3, 1, 1, device="cuda")
    pt = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    call = q4k.paged_attention8
    q = torch.ones(0, 2, 64, dtype=BF16, device="cuda")
    assert call(q, kc, kc, ks, ks, pt, _dev([0, 0, 0]), _dev([3, 0])).shape == (0, 2, 64)
    q = torch.ones(5, 2, 64, dtype=BF16, device="cuda")
    for form in FORMS:
        out = torch.full_like(q, 9.0)
        call(q, kc, kc, ks, ks, pt[:0], _dev([0]), _dev([]), out, form=form)
        assert torch.all(out == 9.0)
        call(q, kc, kc, ks, ks, pt, _dev([0, 0, 3]), _dev([0, 0]), out, form=form)     # positions -3 .. -1: they see nothing
        torch.cuda.synchronize()
        assert not out[:3].any() and torch.all(out[3:] == 9.0)
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,page", [(2, 16), (200, 32)])
def test_wait_runs_out_then_recovers(q4k, form, n, page):
    """As the 16-bit kernels' test: the first copies are awaited for 16 bytes too many, with a bound of 1 ms."""
    g = torch.Generator().manual_seed(n)
    for qt in (F32, BF16):
        if not _takes(form, qt, qt, 64, page, 1.0, 4, 0.0):
            continue
        ((kc, ks, _), (vc, vs, _)), pt = _cache(g, [700, 650], page, 16, 2, 64, I8)
        args = (torch.randn(2 * n, 8, 64, generator=g).to(qt).cuda(), kc, vc, ks, vs, pt.cuda(), _dev([0, n, 2 * n]), _dev([700, 650]))
        want = q4k.paged_attention8(*args, form=form)
        torch.cuda.synchronize()
        assert q4k.device_error_flags() == 0
        t0 = time.time()
        q4k.paged_attention8(*args, wait_limit_us=1000, test_stall=True, form=form)
        torch.cuda.synchronize()
        assert time.time() - t0 < 10.0
        assert q4k.device_error_flags() == 8
        q4k.device_error_clear()
        assert torch.equal(q4k.paged_attention8(*args, form=form), want)
        torch.cuda.synchronize()
        assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("n,qt", [(1, F32), (60, BF16)])
def test_chain(q4k, n, qt):
    """Norm and rotation, append, attention and reading back in a row, plain, as programmatic dependents and in a graph:
    the same bits; and what attention gives is what the values read back give in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(8)
    H, KH, D, page, lens = 8, 2, 64, 16, [n + 200, n]
    pt = torch.randperm(40, generator=g, device="cuda").to(torch.int32).view(2, 20)
    start, ln = _dev([0, n, 2 * n]), _dev(lens)
    q, k, v = (torch.randn(2 * n, h, D, generator=g, device="cuda").to(qt) for h in (H, KH, KH))
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    table = q4k.rope_table(400, D)
    base = [torch.randint(-127, 128, (40, page, KH, D), generator=g, device="cuda").to(I8) for _ in range(2)] + \
        [torch.rand(40, 4, KH, generator=g, device="cuda") * 0.02 for _ in range(2)]

    def chain(cache, pdl):
        a = q4k.kv_append8(k, v, *cache, pt, start, ln, table=table, q=q, q_weight=w, k_weight=w, pdl=pdl)
        y = q4k.paged_attention8(a, *cache, pt, start, ln, pdl=pdl)
        z, _ = q4k.norm_rope(y, q_weight=w, pdl=pdl)
        return a, y, z, *q4k.kv_read8(*cache, pt, start, ln, 2 * n, pdl=pdl, dtype=F32)

    want = chain([t.clone() for t in base], False)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(chain([t.clone() for t in base], True), want))
    cache, graph = [t.clone() for t in base], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(cache, True)
    for _ in range(2):
        for t, b in zip(cache, base):
            t.copy_(b)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    every = _dev([0, lens[0], lens[0] + lens[1]])
    kv = q4k.kv_read8(*cache, pt, every, ln, sum(lens), dtype=F32)
    keys, vals = ([t[:lens[0]].cpu(), t[lens[0]:].cpu()] for t in kv)
    ref, _, bound = plain.attention(want[0].cpu(), keys, vals, dict(new=[n, n], len=lens), 0.125, parts=qt == F32, cache_dtype=F16,
                                    out_dtype=qt)
    # the values read back are rounded to fp32 (2^-24 of themselves, as much in every score)
    size = torch.einsum("hd,jhd->hj", want[0].cpu().double().abs().amax(0), keys[0].double().abs().repeat_interleave(H // KH, 1)).amax() / 8
    bound = bound + _floor(cache[3], cache[1], lens, qt == BF16)
    if qt == BF16:
        bound = bound + _products(want[0].cpu(), [t.double() for t in keys], [t.double() for t in vals], dict(new=[n, n], len=lens),
                                  0.125, None, 0.0)[0]
    assert ((want[1].double().cpu() - ref).abs() <= bound + 2.0 ** -23 * (1 + 2 * size) * max(x.abs().max() for x in vals)).all()
    assert q4k.device_error_flags() == 0


def test_refusals(q4k):
    q = torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    kc, ks = torch.zeros(3, 16, 2, 64, dtype=I8, device="cuda"), torch.zeros(3, 2, 2, device="cuda")
    pt = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    ok = (q, kc, kc, ks, ks, pt, _dev([0, 2]), _dev([2]))
    call = q4k.paged_attention8
    assert not call(*ok).any()

    def swap(i, v):
        return ok[:i] + (v,) + ok[i + 1:]

    for bad, err in [(lambda: call(*swap(0, q.double())), TypeError), (lambda: call(*swap(0, q[:, :3])), ValueError),
                     (lambda: call(*swap(1, kc.to(BF16))), TypeError), (lambda: call(*swap(1, kc.view(torch.uint8))), TypeError),
                     (lambda: call(*swap(2, kc.view(E4M3))), TypeError), (lambda: call(*swap(2, kc[:2])), ValueError),
                     (lambda: call(*swap(3, ks.half())), TypeError), (lambda: call(*swap(3, ks[:2])), ValueError),
                     (lambda: call(*swap(4, ks[:, :1])), ValueError), (lambda: call(*swap(4, ks[..., :1])), ValueError),
                     (lambda: call(*swap(3, ks.cpu())), ValueError), (lambda: call(*swap(5, pt.long())), TypeError),
                     (lambda: call(q, kc, kc, ks[:, :0], ks[:, :0], *ok[5:]), ValueError),
                     (lambda: call(*ok, q[:1]), ValueError), (lambda: call(*ok, window=-1), q4k.Q4KError),
                     (lambda: call(*ok, softcap=math.inf), q4k.Q4KError), (lambda: call(*ok, form="other"), ValueError),
                     (lambda: q4k.paged_attention(q, kc, kc, *ok[5:]), TypeError),
                     (lambda: call(q, kc.to(BF16), kc.to(BF16), ks, ks, *ok[5:]), TypeError)]:
        with pytest.raises(err):
            bad()
    for page, blocks in ((48, 1), (12, 4), (256, 1)):     # blocks of 48, 3 and 256 tokens
        c, s = torch.zeros(3, page, 2, 64, dtype=I8, device="cuda"), torch.zeros(3, blocks, 2, device="cuda")
        with pytest.raises(ValueError):
            call(q, c, c, s, s, *ok[5:])
    odd = torch.zeros(3, 16, 2, 72, dtype=I8, device="cuda")[..., :64]     # rows that are not 16-byte aligned
    with pytest.raises(q4k.Q4KError) as e:
        call(*swap(1, odd))
    assert e.value.status == 2
    for D in (8, 72, 264, 272):
        z = torch.zeros(3, 16, 2, D, dtype=I8, device="cuda")
        with pytest.raises(q4k.Q4KError) as e:
            call(torch.zeros(2, 4, D, dtype=BF16, device="cuda"), z, z, ks, ks, *ok[5:])
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
