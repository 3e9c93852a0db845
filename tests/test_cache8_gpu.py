"""GPU parity of the head norms with the rotation, the append to an 8-bit cache and the way back, against their
definitions in 64 bits."""
import copy

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402
import plain_cache8 as plain8     # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn
EPS = 1e-6


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


def _close(got, ref, bound, what):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound).max()):.3g} x the bound"


def _rounded(ref, err, dtype):
    return err + plain.UNIT[dtype] * (ref.abs() + err) + plain.TINY[dtype]


def _normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, dtype=torch.float64).to(dtype)


# ---------------------------------------------------------------- norms and rotation

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T,H,KH,D,rot", [(1, 32, 8, 128, 128), (3, 5, 1, 64, 32), (17, 2, 2, 80, 80), (2, 1, 1, 256, 64),
                                          (33, 40, 0, 96, 48), (5, 2, 1, 128, 0), (4, 3, 3, 24, 2), (7, 4, 2, 8, 6),
                                          (300, 28, 4, 136, 136)])
def test_norm_rope(q4k, T, H, KH, D, rot, xt, yt, interleaved):
    g = torch.Generator().manual_seed(T * 1000 + D)
    q, k = _normal(g, T, H, D, dtype=xt), _normal(g, T, KH, D, dtype=xt) * 3 if KH else None
    wq, wk = 1 + 0.3 * _normal(g, D), 1 + 0.3 * _normal(g, KH, D) if KH else None
    tab = plain.table(300, rot) if rot else None
    pos = torch.randint(0, 300, (T,), generator=g).to(torch.int32)
    c = lambda t: None if t is None else t.cuda()
    yq, yk = q4k.norm_rope(q.cuda(), c(k), _dev(pos), c(tab), c(wq), c(wk), eps=EPS, interleaved=interleaved, out_dtype=yt)
    assert yq.dtype == yt and (yk is None) == (KH == 0)
    for x, w, y in ((q, wq, yq), (k, wk, yk)):
        if x is None:
            continue
        ref, err = plain8.heads(x, w, EPS, tab[pos.long()] if rot else None, interleaved)
        _close(y, ref, _rounded(ref, err, yt), "norm_rope")
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_norm_rope_strides_in_place(q4k, dtype, pad):
    g = torch.Generator().manual_seed(5 + pad)
    T, H, D = 6, 4, 64
    tab, pos = plain.table(50, D), torch.arange(T, dtype=torch.int32) * 7
    buf = _normal(g, H, T, D + pad, dtype=dtype).cuda()
    wbuf = (1 + 0.3 * _normal(g, D + pad)).cuda()
    x, w = buf.transpose(0, 1)[..., :D], wbuf[pad:]
    ref, err = plain8.heads(x.cpu(), w.cpu(), EPS, tab[pos.long()], False)
    y = torch.full((T, H, D + 2 * pad), 7.0, dtype=dtype, device="cuda")
    out, _ = q4k.norm_rope(x, None, _dev(pos), tab.cuda(), w, q_out=y[..., pad:pad + D], eps=EPS)
    _close(out, ref, _rounded(ref, err, dtype), "strided")
    assert torch.all(y[..., :pad] == 7.0) and torch.all(y[..., pad + D:] == 7.0)
    margin = buf[..., D:].clone()
    out, _ = q4k.norm_rope(x, None, _dev(pos), tab.cuda(), w, q_out=x, eps=EPS)
    assert out.data_ptr() == x.data_ptr()
    _close(x, ref, _rounded(ref, err, dtype), "in place")
    assert torch.equal(buf[..., D:], margin)


def test_norm_without_rotation_or_weight(q4k):
    """Only what is given: no table, no weight (a plain copy and conversion), one tensor normed and not the other."""
    g = torch.Generator().manual_seed(1)
    q, k, w = _normal(g, 9, 3, 128), _normal(g, 9, 2, 128), 1 + 0.3 * _normal(g, 128)
    yq, yk = q4k.norm_rope(q.cuda(), k.cuda(), q_weight=w.cuda(), eps=EPS)
    ref, err = plain8.heads(q, w, EPS, None, False)
    _close(yq, ref, _rounded(ref, err, F32), "normed")
    assert torch.equal(yk.cpu(), k)
    yq, yk = q4k.norm_rope(q.cuda(), k.cuda(), out_dtype=BF16)
    assert torch.equal(yq.cpu(), q.bfloat16()) and torch.equal(yk.cpu(), k.bfloat16())


def test_norm_of_zeros_and_sizes(q4k):
    """A head of zeros is zero with eps > 0; large and small heads come to the same size."""
    w = torch.ones(128, device="cuda")
    x = torch.zeros(4, 1, 128, device="cuda")
    x[1], x[2], x[3] = 1e15, -1e-15, 3.0
    y, _ = q4k.norm_rope(x, q_weight=w, eps=1e-35)
    assert not y[0].any()
    assert torch.allclose(y[1:].abs(), torch.ones(3, 1, 128, device="cuda"), rtol=1e-5)


def test_norm_rope_bad_positions(q4k):
    g = torch.Generator().manual_seed(2)
    x, tab = _normal(g, 5, 2, 64).cuda(), plain.table(10, 64).cuda()
    y = torch.full_like(x, 7.0)
    q4k.norm_rope(x, None, _dev([1, 10, 3, -1, 9]), tab, torch.ones(64, device="cuda"), q_out=y)
    assert q4k.device_error_flags() == 4
    q4k.device_error_clear()
    assert torch.all(y[[1, 3]] == 7.0) and not (y[[0, 2, 4]] == 7.0).any()


# ---------------------------------------------------------------- append

def _append(q4k, cache, new, past, H=3, rot=None, xt=F32, normed=True, interleaved=False, with_q=True, seed=0, pos=None,
            scale_x=1.0, gap=0):
    """Appends to a Cache, checks everything, returns the Cache after."""
    g = torch.Generator().manual_seed(seed)
    _, _, KH, D = cache.codes[0].shape
    rot = D // 2 * 2 if rot is None else rot
    T = sum(new) + gap
    k, v, q = (_normal(g, T, h, D) * scale_x for h in (KH, KH, H))
    k, v, q = k.to(xt), v.to(xt), q.to(xt)
    wk, wq = (1 + 0.3 * _normal(g, D) if normed else None for _ in range(2))
    lens = [n + p for n, p in zip(new, past)]
    tab = plain.table(max(lens + [1]) + 5, rot) if rot else None
    start = [sum(new[:i]) for i in range(len(new) + 1)]
    c = lambda t: None if t is None else t.cuda()
    dev = cache.device()
    q_out = q4k.kv_append8(c(k), c(v), *dev, _dev(start), _dev(lens), table=c(tab), interleaved=interleaved, pos=_dev(pos),
                           q=c(q) if with_q else None, q_weight=c(wq) if with_q else None, k_weight=c(wk), eps=EPS)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    after = copy.copy(cache)
    after.codes, after.scales = [t.cpu() for t in dev[:2]], [t.cpu() for t in dev[2:4]]
    after.touched, after.blocks = [set(), set()], [set(), set()]
    for b, (n, p) in enumerate(zip(new, past)):
        rows = slice(start[b], start[b + 1])
        at = torch.arange(p, p + n) if pos is None else torch.as_tensor(pos)[rows].long()
        cs = tab[at] if rot else None
        x, err = plain8.heads(k[rows], wk, EPS, cs, interleaved)
        plain8.check_append(cache, after, 0, b, x, err, p)
        plain8.check_append(cache, after, 1, b, v[rows].double(), torch.zeros(n, KH, D, dtype=torch.float64), p)
        if with_q:
            ref, err = plain8.heads(q[rows], wq, EPS, cs, interleaved)
            _close(q_out[rows], ref, _rounded(ref, err, xt), "q")
    plain8.check_rest(cache, after)
    return after


@pytest.mark.parametrize("dtype", [I8, E4M3])
@pytest.mark.parametrize("page,block", [(1, 1), (5, 1), (16, 1), (16, 2), (16, 4), (24, 8), (16, 16), (48, 16), (64, 32), (64, 64),
                                        (128, 128), (256, 64)])
def test_append_blocks(q4k, dtype, page, block):
    """Sequences that begin and end inside a block, fill one, cross pages, bring nothing."""
    new, past = [1, 7, 0, 40, 16, 129], [0, 37, 20, 50, 16, 3]
    cache = plain8.Cache(new, 200, page, block, 2, 64, dtype, seed=page + block)
    _append(q4k, cache, new, past)


@pytest.mark.parametrize("dtype", [I8, E4M3])
@pytest.mark.parametrize("KH,H,D,rot,inter", [(1, 1, 8, 8, False), (4, 28, 128, 128, False), (8, 8, 128, 64, True),
                                              (2, 3, 24, 6, False), (1, 2, 72, 10, True), (3, 3, 136, 136, False),
                                              (2, 4, 256, 256, True), (2, 2, 256, 32, False), (2, 2, 80, 0, False)])
@pytest.mark.parametrize("xt", [F32, F16, BF16])
def test_append_heads(q4k, dtype, KH, H, D, rot, inter, xt):
    new, past = [3, 30], [9, 0]
    for block in (1, 16, 64):
        cache = plain8.Cache(new, 64, 64, block, KH, D, dtype, seed=D)
        _append(q4k, cache, new, past, H, rot, xt, interleaved=inter)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("normed,with_q", [(False, True), (True, False), (False, False)])
def test_append_options(q4k, first, normed, with_q):
    new, past = [5, 20], [30, 3]
    cache = plain8.Cache(new, 64, 16, 4, 2, 64, I8, heads_first=first)
    _append(q4k, cache, new, past, normed=normed, with_q=with_q, xt=BF16, pos=[7, 0, 3, 3, 9] + list(range(23)), gap=3)


def test_append_large(q4k):
    """Enough tokens for several rows a thread on the queries' side."""
    new, past = [700, 1, 300], [5, 100, 0]
    for block, D in ((16, 128), (128, 256)):
        cache = plain8.Cache(new, 720, 128, block, 2, D, I8, seed=D)
        _append(q4k, cache, new, past, H=16, xt=BF16)


@pytest.mark.parametrize("dtype", [I8, E4M3])
@pytest.mark.parametrize("block", [1, 4, 32])
def test_append_step_by_step(q4k, dtype, block):
    """Tokens one by one and a few at a time, of growing size: the block's scale grows and its codes follow; then the same
    positions again from the middle of a block (drafted tokens taken back)."""
    cache = plain8.Cache([0, 0], 64, 32, block, 2, 64, dtype)
    past = [0, 17]
    for step, n in enumerate([1, 1, 2, 1, 5, 1, 1, 3, 9]):
        cache = _append(q4k, cache, [n, 1], past, seed=step, scale_x=1.3 ** step)
        past = [past[0] + n, past[1] + 1]
    back = [past[0] - 6, past[1] - 1]
    _append(q4k, cache, [3, 1], back, seed=99, scale_x=0.1)


def test_append_values_off_the_scale(q4k):
    """Zeros, the smallest and largest numbers, infinities and NaN."""
    big = torch.finfo(F32).max
    rows = torch.zeros(7, 1, 64)
    rows[1, 0, :2] = torch.tensor([big, -big])
    rows[2, 0, :2] = torch.tensor([1e-45, -1e-40])
    rows[3, 0, :4] = torch.tensor([float("inf"), float("-inf"), 1.0, -2.0])
    rows[4, 0, :3] = torch.tensor([float("nan"), 3.0, 1.5])
    rows[5, 0, :] = float("inf")
    rows[6, 0, :] = float("nan")
    for dtype in (I8, E4M3):
        top = plain8.TOP[dtype]
        cache = plain8.Cache([7], 16, 16, 1, 1, 64, dtype)
        dev = cache.device()
        q4k.kv_append8(rows.cuda(), rows.cuda(), *dev, _dev([0, 7]), _dev([7]))
        assert q4k.device_error_flags() == 0
        for side in (0, 1):
            page = int(cache.table[0, 0])
            c = dev[side][page, :7, 0].cpu().float()
            s = dev[2 + side][page, :7, 0].cpu()
            assert not c[0].any() and s[0] == 2.0 ** -126
            assert c[1, 0] == top and c[1, 1] == -top and s[1] == torch.tensor(big) / torch.tensor(top)
            # 1e-40 2^126 = 0.0085: 0 in int8, 4 steps of 2^-9 in e4m3
            assert s[2] == 2.0 ** -126 and c[2, 0] == 0 and c[2, 1] == (0.0 if dtype == I8 else -2.0 ** -7)
            assert c[3, 0] == top and c[3, 1] == -top and c[3, 3] == -top and s[3] == torch.tensor(2.0) / torch.tensor(top)
            assert c[4, 1] == top and (torch.isnan(c[4, 0]) if dtype == E4M3 else c[4, 0] == 0)
            assert torch.all(c[5] == top) and s[5] == 2.0 ** -126
            assert torch.all(torch.isnan(c[6]) if dtype == E4M3 else c[6] == 0) and s[6] == 2.0 ** -126


def test_append_bad_indices(q4k):
    """Pages, positions and lengths outside the buffers are not followed; the other sequence's tokens arrive."""
    g = torch.Generator().manual_seed(4)
    k = _normal(g, 6, 2, 64)
    for what in ("page", "length", "short", "capacity", "starts", "row"):
        cache = plain8.Cache([3, 3], 32, 16, 16, 2, 64, I8)
        dev = cache.device()
        start, lens, kw = [0, 3, 6], [10, 20], {}
        if what == "page":
            dev[4][0, 0] = 99
        elif what == "length":
            lens[0] = -5
        elif what == "short":
            lens[0] = 2
        elif what == "capacity":
            lens[0] = 2 ** 31 - 1
        elif what == "starts":
            start = [-3, 3, 6]
        else:
            kw = dict(table=plain.table(4, 64).cuda(), pos=_dev([0, 4, -1, 1, 2, 3]))
        q4k.kv_append8(k.cuda(), k.cuda(), *dev, _dev(start), _dev(lens), **kw)
        torch.cuda.synchronize()
        assert q4k.device_error_flags() == 4, what
        q4k.device_error_clear()
        pages = [int(p) for p in cache.table[1, 1:2]]
        for side in (0, 1):
            moved = (cache.codes[side] != dev[side].cpu()).any(-1).any(-1).nonzero()
            good = set(pages) | ({int(cache.table[0, 0])} if what == "row" else set())
            assert {int(p) for p, _ in moved} <= good, what
            assert int(pages[0]) in {int(p) for p, _ in moved}, what


# ---------------------------------------------------------------- reading back

@pytest.mark.parametrize("dtype", [I8, E4M3])
@pytest.mark.parametrize("yt", [F32, F16, BF16])
@pytest.mark.parametrize("page,block,KH,D,first", [(16, 16, 4, 128, False), (5, 1, 1, 8, False), (64, 64, 2, 256, True),
                                                   (48, 8, 3, 72, True), (1, 1, 2, 64, False), (128, 128, 1, 136, False)])
def test_read(q4k, dtype, yt, page, block, KH, D, first):
    lens, take = [1, 130, 20, 77], [1, 130, 0, 33]
    cache = plain8.Cache(lens, 130, page, block, KH, D, dtype, seed=D, heads_first=first)
    start = [2] + [2 + sum(take[:i + 1]) for i in range(4)]
    k = torch.full((start[-1] + 3, KH, D), 7.0, dtype=yt, device="cuda")
    v = torch.full_like(k, 7.0)
    out = q4k.kv_read8(*cache.device(), _dev(start), _dev(lens), k.shape[0], k, v)
    assert out[0].data_ptr() == k.data_ptr() and q4k.device_error_flags() == 0
    for side, y in enumerate((k, v)):
        assert torch.all(y[:2] == 7.0) and torch.all(y[start[-1]:] == 7.0)
        for b, n in enumerate(take):
            want = cache.values(side, b, torch.arange(lens[b] - n, lens[b])).float().to(yt)   # exact in 64 bits, rounded to fp32 first
            assert torch.equal(y[start[b]:start[b + 1]].cpu(), want)


def test_read_strides(q4k):
    """Outputs of any strides, among them ones that no wide store fits, and codes that are not aligned."""
    cache = plain8.Cache([40], 40, 16, 4, 2, 64, I8)
    for pad in (1, 8):
        buf = torch.full((2, 40, 64 + pad), 7.0, dtype=BF16, device="cuda")
        k, v = buf.transpose(0, 1)[..., :64], torch.empty(40, 2, 64, dtype=BF16, device="cuda")
        dev = cache.device()
        wide = torch.zeros(*dev[0].shape[:3], 64 + pad, dtype=I8, device="cuda")
        wide[..., pad:] = dev[0]
        q4k.kv_read8(wide[..., pad:], *dev[1:], _dev([0, 40]), _dev([40]), 40, k, v)
        for side, y in enumerate((k, v)):
            assert torch.equal(y.cpu(), cache.values(side, 0, torch.arange(40)).float().to(BF16))
        assert torch.all(buf[..., 64:] == 7.0)


def test_read_bad_indices(q4k):
    cache = plain8.Cache([20, 20], 32, 16, 16, 2, 64, I8)
    dev = cache.device()
    dev[4][0, 1] = -1
    k, v = torch.full((40, 2, 64), 7.0, device="cuda"), torch.full((40, 2, 64), 7.0, device="cuda")
    q4k.kv_read8(*dev, _dev([0, 20, 40]), _dev([20, 20]), 40, k, v)
    assert q4k.device_error_flags() == 4
    q4k.device_error_clear()
    assert torch.all(k[16:20] == 7.0) and torch.all(v[16:20] == 7.0)
    assert torch.equal(k[20:].cpu(), cache.values(0, 1, torch.arange(20)).float())
    assert torch.equal(k[:16].cpu(), cache.values(0, 0, torch.arange(16)).float())


# ---------------------------------------------------------------- streams and graphs

def test_captured_and_replayed(q4k):
    """Append and read in one graph, as programmatic dependents, follow the lengths on the device."""
    cache = plain8.Cache([0, 0], 64, 16, 4, 2, 64, I8)
    dev, eager = cache.device(), cache.device()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 2, 64, generator=g, device="cuda")
    start, lens = _dev([0, 1, 2]), _dev([1, 30])
    tab = plain.table(64, 64).cuda()
    w = torch.ones(64, device="cuda")

    def step(c, n):
        q = q4k.kv_append8(x, x, *c, start, n, table=tab, q=x, k_weight=w, q_weight=w, pdl=True)
        return q, *q4k.kv_read8(*c, start, n, 2, pdl=True)

    step(cache.device(), lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(dev, lens)
    for i in range(5):
        x.copy_(torch.randn(2, 2, 64, generator=g, device="cuda") * (i + 1))
        graph.replay()
        want = step(eager, lens)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(dev[:4], eager[:4]))
        lens += 1
    assert q4k.device_error_flags() == 0


def test_given_stream(q4k):
    cache = plain8.Cache([40], 40, 16, 16, 2, 64, I8)
    dev = cache.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k, v = q4k.kv_read8(*dev, _dev([0, 40]), _dev([40]), 40, stream=side, dtype=F32)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(k.cpu(), cache.values(0, 0, torch.arange(40)).float())
    assert torch.equal(v.cpu(), cache.values(1, 0, torch.arange(40)).float())


def test_empty_calls(q4k):
    cache = plain8.Cache([1], 16, 16, 16, 2, 64, I8)
    dev = cache.device()
    none = torch.zeros(0, 2, 64, device="cuda")
    assert q4k.kv_append8(none, none, *dev, _dev([0, 0]), _dev([5])) is None
    k, v = q4k.kv_read8(*dev, _dev([0, 0]), _dev([5]), 0)
    assert k.shape == (0, 2, 64) and k.dtype == BF16
    q, k = q4k.norm_rope(none, none)
    assert q.shape == k.shape == (0, 2, 64)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dev[:4], cache.codes + cache.scales))
    assert q4k.device_error_flags() == 0
