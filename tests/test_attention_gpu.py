"""GPU parity of attention over a paged cache against its definition in 64 bits: head layouts, lengths, page sizes,
masks, types.  Every cache slot that holds no position is NaN, and every unused page table entry is -1."""
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


def _dev(x):
    return None if x is None else torch.as_tensor(x, dtype=torch.int32).cuda()


def _run(q4k, case, H, KH, D, page, qt=BF16, ct=BF16, ot=None, softcap=0.0, slopes=None, first=False, scale=None,
         std=1.5, seed=0, spare=2):
    """Builds the call, checks out and lse, returns (out, the call)."""
    ot = qt if ot is None else ot
    g = torch.Generator().manual_seed(seed * 7919 + sum(case["len"]) * 31 + H * D)
    T = sum(case["new"])
    q = (torch.randn(T, H, D, generator=g, dtype=torch.float64) * std).to(qt)
    keys = [torch.randn(n, KH, D, generator=g).to(ct) for n in case["len"]]
    vals = [torch.randn(n, KH, D, generator=g).to(ct) for n in case["len"]]
    order = torch.randperm(sum(-(-n // page) for n in case["len"]) + spare, generator=g)
    kc, pt = plain.paged(keys, page, ct, order, spare, heads_first=first)
    vc, _ = plain.paged(vals, page, ct, order, spare, heads_first=first)
    if case.get("window") and case.get("free"):     # pages that no window reaches any more
        for b, (n, length) in enumerate(zip(case["new"], case["len"])):
            pt[b, :max(0, length - n + 1 - case["window"]) // page] = -1
    kc = kc.cuda() if not first else kc.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    vc = vc.cuda() if not first else vc.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    start = _dev([sum(case["new"][:i]) for i in range(len(case["new"]) + 1)])
    lse = torch.full((T, H), 7.0, device="cuda")
    sl = None if slopes is None else torch.tensor(slopes, dtype=F32)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    args = (q.cuda(), kc, vc, pt.cuda(), start, _dev(case["len"]))
    kw = dict(scale=scale, out_dtype=ot, softcap=softcap, slopes=None if sl is None else sl.cuda(),
              window=case.get("window", 0), causal=case.get("causal", True), prefix_len=_dev(case.get("prefix")),
              kv_start=_dev(case.get("kv_start")))
    out = q4k.paged_attention(*args, lse=lse, **kw)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    assert out.dtype == ot and tuple(out.shape) == (T, H, D)
    many = qt != ct or ot == F32
    ref, rl, bound = plain.attention(q, keys, vals, case, scale, softcap, sl, many, ct, ot)
    err = (out.double().cpu() - ref).abs()
    assert (err <= bound).all(), f"out: worst {float((err / bound).max()):.3g} x the bound"
    dead = torch.isinf(rl)
    got = lse.double().cpu()
    assert torch.equal(dead, torch.isinf(got) & (got < 0))
    assert not out.cpu()[dead].any(), "a row that sees nothing is zero"
    # the scores' own errors (bounded well inside 2^-12 here) and fp32's on the sum
    tol = 2.0 ** -12 + 2.0 ** -20 * rl[~dead].abs()
    assert ((got[~dead] - rl[~dead]).abs() <= tol).all()
    return out, lambda **over: q4k.paged_attention(*args, **{**kw, **over})


TYPES = [(BF16, BF16, BF16), (F16, F16, F16), (F32, BF16, F32), (F32, F16, F32), (BF16, BF16, F32), (F16, F16, BF16),
         (F32, BF16, BF16), (BF16, F16, BF16)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("new,lens,H,KH,D,page", [
    ([1], [1], 28, 4, 128, 16),
    ([1, 1, 1], [300, 17, 128], 28, 4, 128, 16),
    ([5, 5], [40, 261], 28, 4, 128, 16),
    ([1, 0, 40, 3], [9, 12, 200, 3], 8, 8, 64, 32),
    ([70], [333], 6, 2, 128, 64),
])
def test_types(q4k, new, lens, H, KH, D, page, types):
    _run(q4k, dict(new=new, len=lens), H, KH, D, page, *types)


@pytest.mark.parametrize("H,KH,D", [(1, 1, 8), (4, 4, 16), (8, 1, 64), (32, 1, 128), (9, 3, 80), (5, 5, 96), (16, 2, 112),
                                    (7, 1, 136), (4, 2, 192), (16, 4, 256), (40, 1, 64)])
@pytest.mark.parametrize("many", [False, True])
def test_heads_and_dims(q4k, H, KH, D, many):
    case = dict(new=[1, 4, 37], len=[200, 65, 131])
    _run(q4k, case, H, KH, D, 16, F32 if many else BF16, BF16)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 48, 64, 100, 128, 256, 512])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, F16, F32)])
def test_page_sizes(q4k, page, first, types):
    _run(q4k, dict(new=[1, 150, 2], len=[513, 277, 2]), 14, 2, 128, page, *types, first=first)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("past", [0, 1, 100])
def test_lengths(q4k, n, past):
    _run(q4k, dict(new=[n], len=[n + past]), 4, 2, 64, 16, seed=n)


MASKS = [
    dict(window=1), dict(window=16), dict(window=100, free=True), dict(causal=False), dict(causal=False, window=30),
    dict(prefix=[50, 0, 1000, 3]), dict(prefix=[5, 300, 0, 0], window=20),
    dict(kv_start="docs"), dict(kv_start="docs", prefix=[10, 40, 0, 200]), dict(kv_start="beyond"),
    dict(kv_start="docs", causal=False, window=7),
]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("H,KH,D,page,types", [(4, 2, 128, 16, (BF16, BF16, BF16)), (14, 2, 64, 32, (F16, F16, F16)),
                                               (7, 1, 96, 5, (F32, BF16, F32)), (3, 3, 128, 64, (F32, F16, F32))])
def test_masks(q4k, mask, H, KH, D, page, types):
    case = dict(new=[90, 1, 20, 3], len=[300, 130, 20, 260], **mask)
    if mask.get("kv_start"):
        starts = []
        for n, length in zip(case["new"], case["len"]):
            for i in range(n):
                p = length - n + i
                if mask["kv_start"] == "docs":
                    starts.append(p // 37 * 37)
                else:       # every third token sees nothing, one far past the end, one negative
                    starts.append(10 ** 9 if i % 3 == 0 else (-5 if i % 3 == 1 else p))
        case["kv_start"] = starts
    _run(q4k, case, H, KH, D, page, *types)


@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F16, F16, F16), (F32, BF16, F32), (F32, F16, F32)])
@pytest.mark.parametrize("softcap,biased,causal", [(30.0, False, True), (0.0, True, True), (50.0, True, True),
                                                   (5.0, True, False)])
def test_cap_and_bias(q4k, types, softcap, biased, causal):
    H = 8
    slopes = [2.0 ** (-i - 1) for i in range(H)] if biased else None
    _run(q4k, dict(new=[1, 100, 6], len=[400, 150, 70], causal=causal), H, 4, 128, 16, *types, softcap=softcap,
         slopes=slopes, std=4.0)


@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, BF16, F32), (F32, F16, F32)])
@pytest.mark.parametrize("new,lens", [([1], [20000]), ([3, 1], [5000, 9001]), ([130], [6000])])
def test_long(q4k, new, lens, types):
    """Rows split over many CTAs."""
    _run(q4k, dict(new=new, len=lens), 8, 2, 128, 64, *types)


def test_many_sequences(q4k):
    """More sequences than the kernels keep in shared memory, many of them without tokens."""
    n = 1300
    new = [(b % 3) * (b % 2) for b in range(n)]
    lens = [new[b] + b % 40 for b in range(n)]
    _run(q4k, dict(new=new, len=lens), 2, 1, 64, 16)
    _run(q4k, dict(new=new, len=lens), 2, 1, 64, 16, F32, F16, F32)


@pytest.mark.parametrize("std", [1e-3, 40.0])
@pytest.mark.parametrize("types", [(F32, F16, F32), (F32, BF16, F32), (BF16, BF16, BF16)])
def test_flat_and_peaked_scores(q4k, std, types):
    _run(q4k, dict(new=[1, 33], len=[150, 260]), 4, 2, 128, 16, *types, std=std)


def test_scores_off_the_scale(q4k):
    """Infinite and NaN keys: a masked one changes nothing, a score of -inf drops its key, all of them give a zero row."""
    D, page = 64, 16
    k = torch.randn(20, 1, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    v = torch.randn(20, 1, D, generator=torch.Generator().manual_seed(2)).to(BF16)
    k[5] = -math.inf
    for qt, ot in ((BF16, BF16), (F32, F32)):
        for n in (1, 15):
            q = torch.rand(n, 1, D, generator=torch.Generator().manual_seed(3)).to(qt) + 0.5
            kc, pt = plain.paged([k], page, BF16, torch.arange(4))
            vc, _ = plain.paged([v], page, BF16, torch.arange(4))
            kc, vc, pt, qd = kc.cuda(), vc.cuda(), pt.cuda(), q.cuda()
            start, ln = _dev([0, n]), _dev([20])
            out = q4k.paged_attention(qd, kc, vc, pt, start, ln)
            lse = torch.zeros(n, 1, device="cuda")
            # without key 5 the same call gives the same rows
            keep = [j for j in range(20) if j != 5]
            k2, _ = plain.paged([k[keep]], page, BF16, torch.arange(4))
            v2, _ = plain.paged([v[keep]], page, BF16, torch.arange(4))
            want = q4k.paged_attention(qd, k2.cuda(), v2.cuda(), pt, start, _dev([19]))
            assert torch.allclose(out.float(), want.float(), atol=2.0 ** -6 if ot == BF16 else 1e-5)
            # NaN key visible to the last token only
            kn = kc.clone()
            kn[pt[0, 1], 3] = math.nan
            o = q4k.paged_attention(qd, kn, vc, pt, start, ln)
            assert torch.isnan(o[-1]).all()
            assert torch.equal(o[:-1], out[:-1])
            # every visible score -inf
            kn = torch.full_like(kc, -math.inf)
            o = q4k.paged_attention(qd, kn, vc, pt, start, ln, lse=lse)
            assert not o.any() and torch.isinf(lse).all() and (lse < 0).all()
    assert q4k.device_error_flags() == 0


def test_strides_streams_and_repeats(q4k):
    """Padded and transposed q and out, keys and values in one buffer, a side stream, a graph; the same bits each time."""
    g = torch.Generator().manual_seed(11)
    for qt in (F32, BF16):
        n, H, KH, D, page = 9, 8, 2, 64, 16
        q = torch.randn(n, H, D, generator=g).to(qt).cuda()
        both = torch.randn(6, 2, page, KH, D, generator=g).to(BF16).cuda()
        pt = torch.tensor([[3, 0, 5], [1, 4, 2]], dtype=torch.int32, device="cuda")
        start, ln = _dev([0, 4, 9]), _dev([40, 33])
        plain_out = q4k.paged_attention(q, both[:, 0].contiguous(), both[:, 1].contiguous(), pt, start, ln)
        wide = torch.full((H, n, D + 16), 3.0, dtype=qt, device="cuda")
        out = wide[..., :D].transpose(0, 1)
        qs = torch.zeros(H, n, D + 8, dtype=qt, device="cuda")[..., :D].transpose(0, 1)
        qs.copy_(q)
        assert q4k.paged_attention(qs, both[:, 0], both[:, 1], pt, start, ln, out) is out
        assert torch.equal(out, plain_out) and torch.all(wide[..., D:] == 3.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o2 = q4k.paged_attention(q, both[:, 0], both[:, 1], pt, start, ln, stream=side)
        side.synchronize()
        assert torch.equal(o2, plain_out)
        graph, o3 = torch.cuda.CUDAGraph(), torch.zeros_like(plain_out)
        with torch.cuda.graph(graph):
            q4k.paged_attention(q, both[:, 0], both[:, 1], pt, start, ln, o3)
        for _ in range(3):
            o3.zero_()
            graph.replay()
            assert torch.equal(o3, plain_out)
        # the captured call follows the lengths on the device
        ln.copy_(_dev([20, 30]))
        graph.replay()
        assert torch.equal(o3, q4k.paged_attention(q, both[:, 0], both[:, 1], pt, start, ln))
    out, again = _run(q4k, dict(new=[1, 64], len=[9000, 3000]), 8, 2, 128, 16)
    for _ in range(3):
        assert torch.equal(again(), out)
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("qt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 40])
def test_offsets_past_32_bits(q4k, n, qt):
    """Pages more than 2^31 elements (and 2^32 bytes) into the cache."""
    KH, D, page = 2, 64, 16
    pages = 2 ** 31 // (KH * D * page) + 40
    kc = torch.empty(pages, page, KH, D, dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    pt = torch.tensor([[pages - 1, 0, pages - 5, 3, pages - 2]], dtype=torch.int32)
    length = 70
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(length, KH, D, generator=g).to(BF16) for _ in range(2))
    for i, p in enumerate(pt[0].tolist()):
        part = slice(16 * i, min(length, 16 * i + 16))
        kc[p, :k[part].shape[0]] = k[part].cuda()
        vc[p, :v[part].shape[0]] = v[part].cuda()
    q = torch.randn(n, 4, D, generator=g).to(qt)
    case = dict(new=[n], len=[length])
    ref, _, bound = plain.attention(q, [k], [v], case, 0.125, parts=qt == F32, out_dtype=qt)
    out = q4k.paged_attention(q.cuda(), kc, vc, pt.cuda(), _dev([0, n]), _dev([length]))
    assert ((out.double().cpu() - ref).abs() <= bound).all()
    assert q4k.device_error_flags() == 0


def test_bad_indices_are_not_followed(q4k):
    """Pages outside the cache, lengths past the page table, rows outside the call: flagged, nothing followed."""
    q = torch.ones(4, 2, 64, dtype=BF16, device="cuda")
    kc = torch.ones(3, 16, 1, 64, dtype=BF16, device="cuda")
    for pt, start, ln in [([[7, 0]], [0, 4], [20]), ([[-1, 0]], [0, 4], [20]), ([[0, 1]], [0, 4], [33]),
                          ([[0, 1]], [0, 9], [20]), ([[0, 1]], [-3, 4], [20]), ([[0, 1], [1, 2]], [0, 4, 2], [20, 20]),
                          ([[0, 1]], [0, 4], [-7])]:
        for x in (q, q.float()):
            q4k.paged_attention(x, kc, kc, *[torch.tensor(v, dtype=torch.int32, device="cuda") for v in (pt, start, ln)])
            torch.cuda.synchronize()
            assert q4k.device_error_flags() == 4, (pt, start, ln)
            q4k.device_error_clear()


def test_nothing_to_do(q4k):
    """No tokens, no sequences, rows of no sequence."""
    kc = torch.ones(3, 16, 1, 64, dtype=BF16, device="cuda")
    pt = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    q = torch.ones(0, 2, 64, dtype=BF16, device="cuda")
    assert q4k.paged_attention(q, kc, kc, pt, _dev([0, 0, 0]), _dev([3, 0])).shape == (0, 2, 64)
    q = torch.ones(5, 2, 64, dtype=BF16, device="cuda")
    out = torch.full_like(q, 9.0)
    q4k.paged_attention(q, kc, kc, pt[:0], _dev([0]), _dev([]), out)
    assert torch.all(out == 9.0)
    q4k.paged_attention(q, kc, kc, pt, _dev([0, 0, 3]), _dev([0, 0]), out)     # positions -3 .. -1: they see nothing
    torch.cuda.synchronize()
    assert not out[:3].any() and torch.all(out[3:] == 9.0)
    assert q4k.device_error_flags() == 0


def test_refusals(q4k):
    q = torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    kc = torch.zeros(3, 16, 2, 64, dtype=BF16, device="cuda")
    pt = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    start, ln = _dev([0, 2]), _dev([2])
    ok = (q, kc, kc, pt, start, ln)
    call = q4k.paged_attention

    def swap(i, v):
        return ok[:i] + (v,) + ok[i + 1:]

    lse = torch.zeros(2, 4, device="cuda")
    for bad, err in [(lambda: call(*swap(0, q.double())), TypeError), (lambda: call(*swap(0, q[0])), ValueError),
                     (lambda: call(*swap(0, q.cpu())), ValueError), (lambda: call(*swap(0, q[:, :3])), ValueError),
                     (lambda: call(*swap(0, q[..., :32])), ValueError), (lambda: call(*swap(1, kc.float())), TypeError),
                     (lambda: call(*swap(2, kc.half())), TypeError), (lambda: call(*swap(2, kc[:2])), ValueError),
                     (lambda: call(*swap(3, pt.long())), TypeError), (lambda: call(*swap(3, pt[0])), ValueError),
                     (lambda: call(*swap(4, start[:1])), ValueError), (lambda: call(*swap(5, ln.cpu())), ValueError),
                     (lambda: call(*ok, q[:1]), ValueError), (lambda: call(*ok, q, out_dtype=F32), TypeError),
                     (lambda: call(*ok, window=-1), q4k.Q4KError), (lambda: call(*ok, softcap=-1.0), q4k.Q4KError),
                     (lambda: call(*ok, softcap=math.inf), q4k.Q4KError), (lambda: call(*ok, scale=math.nan), q4k.Q4KError),
                     (lambda: call(*ok, slopes=lse[0, :3]), ValueError), (lambda: call(*ok, slopes=lse[0].half()), TypeError),
                     (lambda: call(*ok, prefix_len=_dev([1, 2])), ValueError), (lambda: call(*ok, kv_start=_dev([1])), ValueError),
                     (lambda: call(*ok, lse=lse[:1]), ValueError), (lambda: call(*ok, lse=lse.half()), TypeError)]:
        with pytest.raises(err):
            bad()
    # rows that are not 16-byte aligned, and sizes the kernels do not take
    odd = torch.zeros(2, 4, 65, dtype=BF16, device="cuda")[..., :64]
    with pytest.raises(q4k.Q4KError) as e:
        call(*swap(0, odd))
    assert e.value.status == 2
    for D in (12, 264):
        with pytest.raises(q4k.Q4KError) as e:
            z = torch.zeros(3, 16, 2, D, dtype=BF16, device="cuda")
            call(torch.zeros(2, 4, D, dtype=BF16, device="cuda"), z, z, pt, start, ln)
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.7])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, F16, F32)])
def test_scales(q4k, scale, types):
    """Negative, zero and large scales, masked rows among them."""
    for new, lens in (([1], [70]), ([90, 3], [200, 40])):
        _run(q4k, dict(new=new, len=lens, window=33), 4, 2, 64, 16, *types, scale=scale)


@pytest.mark.parametrize("H", [130, 260])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, BF16, F32)])
def test_large_groups(q4k, H, types):
    """More query heads per cache head than half a tile of rows holds, and than a whole one."""
    _run(q4k, dict(new=[3, 1], len=[90, 20]), H, 1, 64, 16, *types)


def test_one_page_table_column_and_empty_cache(q4k):
    """A page table one column wide; no cached position: every row sees nothing; a cache without pages: refused."""
    _run(q4k, dict(new=[1, 5], len=[13, 16]), 4, 2, 64, 16)
    kc = torch.zeros(0, 16, 2, 64, dtype=BF16, device="cuda")
    for dtype, n in ((BF16, 1), (F32, 1), (BF16, 40)):
        q = torch.ones(n, 4, 64, dtype=dtype, device="cuda")
        out = torch.full_like(q, 3.0)
        pt = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
        with pytest.raises(q4k.Q4KError):      # no cache to point at
            q4k.paged_attention(q, kc, kc, pt, _dev([0, n]), _dev([0]), out)
        one = torch.zeros(1, 16, 2, 64, dtype=BF16, device="cuda")
        q4k.paged_attention(q, one, one, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), _dev([0, n]), _dev([0]), out)
        torch.cuda.synchronize()
        assert not out.any()
    assert q4k.device_error_flags() == 0
