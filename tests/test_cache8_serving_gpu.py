"""The 8-bit cache as a serving loop uses it: prompt chunks and single tokens through norms, rotation, append and attention
against 64 bits, captured graphs that share the library's scratch, two streams at once, padded batches, page tables far
wider than the sequences, and the widened form's passes and refusals."""
import copy
import math

import pytest

torch = pytest.importorskip("torch")
import plain_attention as plain   # noqa: E402
import plain_cache8 as plain8     # noqa: E402
from test_attention8_gpu import FORMS, _cache, _floor, _products, _takes   # noqa: E402
from test_cache8_gpu import _append   # noqa: E402

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
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _starts(new):
    return [sum(new[:i]) for i in range(len(new) + 1)]


def _bound(q, keys, vals, case, scale, qt, chunk, vs, vc, slopes=None):
    """64-bit attention over the cache's own values, its log-sum-exp, what a kernel may be off by in each."""
    ref, rl, bound = plain.attention(q, keys, vals, case, scale, 0.0, slopes, qt == F32, F16, qt)
    bound = bound + _floor(vs, vc, case["len"], chunk)
    off = 0.0
    if chunk:
        more, off = _products(q, keys, vals, case, scale, slopes, 0.0)
        bound = bound + more
    return ref, rl, bound, off


@pytest.mark.parametrize("ct,page,block", [(I8, 16, 16), (E4M3, 16, 1), (I8, 48, 4), (E4M3, 128, 128)])
@pytest.mark.parametrize("qt", [F32, BF16])
def test_a_sequence_step_by_step(q4k, ct, page, block, qt):
    """Two sequences fed by ragged chunks, then token by token.  After each step: the append against its definition, the
    attention against 64 bits over the cache as it then is, the read back exactly code times scale."""
    H, KH, D, most = 6, 2, 64, 200
    g = torch.Generator().manual_seed(21)
    cache = plain8.Cache([0, 0], most, page, block, KH, D, ct, seed=4)
    dev = cache.device()
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2))
    tab = plain.table(most, D)
    lens = [0, 0]
    for new in ([33, 70], [40, 1], [0, 65], [1, 1], [1, 1], [3, 0], [1, 1]):
        T = sum(new)
        k, v, q = (torch.randn(T, h, D, generator=g).to(qt) for h in (KH, KH, H))
        past, lens = lens, [a + b for a, b in zip(lens, new)]
        start = _starts(new)
        idx = (dev[4], _dev(start), _dev(lens))
        before = copy.copy(cache)
        a = q4k.kv_append8(k.cuda(), v.cuda(), *dev[:4], *idx, table=tab.cuda(), q=q.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda(), eps=EPS)
        y = q4k.paged_attention8(a, *dev[:4], *idx)
        r = q4k.kv_read8(*dev[:4], *idx, T, dtype=F32)
        torch.cuda.synchronize()
        cache = copy.copy(before)
        cache.codes, cache.scales = [t.cpu() for t in dev[:2]], [t.cpu() for t in dev[2:4]]
        cache.touched, cache.blocks = [set(), set()], [set(), set()]
        for b, (n, p) in enumerate(zip(new, past)):
            rows = slice(start[b], start[b + 1])
            x, err = plain8.heads(k[rows], wk, EPS, tab[p:p + n], False)
            plain8.check_append(before, cache, 0, b, x, err, p)
            plain8.check_append(before, cache, 1, b, v[rows].double(), torch.zeros(n, KH, D, dtype=torch.float64), p)
            for side in (0, 1):
                assert torch.equal(r[side][rows].cpu(), cache.values(side, b, torch.arange(p, p + n)).float())
        plain8.check_rest(before, cache)
        keys, vals = ([cache.values(side, b, torch.arange(n)) for b, n in enumerate(lens)] for side in (0, 1))
        chunk = qt == BF16     # (the choice of the form is the library's)
        ref, _, bound, _ = _bound(a.cpu(), keys, vals, dict(new=new, len=lens), 1 / math.sqrt(D), qt, chunk, cache.scales[1], cache.codes[1])
        assert ((y.double().cpu() - ref).abs() <= bound).all()
        cache.table = before.table
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("ct", [I8, E4M3])
@pytest.mark.parametrize("block,bad", [(4, [0, 4, 9]), (4, [1, 2, 3]), (16, [0]), (16, [3, 4]), (64, [0, 1, 2, 3]), (64, range(40)),
                                       (1, [0, 5])])
def test_tokens_without_a_place_in_a_block(q4k, ct, block, bad):
    """Keys whose rotation row lies outside the table are left out and flagged, wherever in a block they are: the others of it
    get a scale of their own, and a block that gets none keeps its codes and its scale, even one below the least."""
    n, past, KH, D, page = 40, 3, 2, 64, 64
    g = torch.Generator().manual_seed(33)
    cache = plain8.Cache([past + n], past + n, page, block, KH, D, ct, seed=7)
    for s in cache.scales:
        s[cache.table[0, 0].long(), 0] = 1e-39 if len(bad) == n else 1e-3
    dev = cache.device()
    k, v = (torch.randn(n, KH, D, generator=g) for _ in range(2))
    tab = plain.table(64, D)
    pos = torch.arange(past, past + n)
    pos[list(bad)] = 10 ** 6
    q4k.kv_append8(k.cuda(), v.cuda(), *dev[:4], dev[4], _dev([0, n]), _dev([past + n]), table=tab.cuda(), pos=_dev(pos))
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 4
    q4k.device_error_clear()
    after = copy.copy(cache)
    after.codes, after.scales = [t.cpu() for t in dev[:2]], [t.cpu() for t in dev[2:4]]
    after.touched, after.blocks = [set(), set()], [set(), set()]
    plain8.check_append(cache, after, 1, 0, v.double(), torch.zeros(n, KH, D, dtype=torch.float64), past)
    good = [i for i in range(n) if i not in bad]
    x, err = plain8.heads(k[good], None, EPS, tab[torch.tensor(good, dtype=torch.long) + past], False)
    for first in range(0, past + n, block):
        here = [j for j, i in enumerate(good) if first <= past + i < first + block]
        at = [past + good[j] for j in here]
        old = list(range(first, min(first + block, past)))
        pg, slot = cache.where(0, [first])
        was, got = (c.scales[0][int(pg), int(slot) // block].double() for c in (cache, after))
        every = torch.arange(first, min(first + block, past + n))
        if not here:
            assert torch.equal(was, got)
            where = cache.where(0, every)
            assert torch.equal(*(c.codes[0].view(torch.uint8)[where] for c in (cache, after)))
            continue
        want = (x[here].abs().amax((0, 2)) / plain8.TOP[ct]).clamp(min=plain8.LEAST)
        want = torch.maximum(want, was) if old else want
        assert ((got - want).abs() <= err[here].amax((0, 2)) / plain8.TOP[ct] + 2.0 ** -23 * want).all()
        y = x[here] / got[:, None]
        off = (after.values(0, 0, at) / got[:, None] - y).abs()
        near = plain8.half_step(y * (1 + 2.0 ** -20), ct) * (1 + 2.0 ** -20) + err[here] / got[:, None] + y.abs() * 2.0 ** -22
        assert (off <= near).all()


@pytest.mark.parametrize("dtype,block", [(I8, 64), (E4M3, 128)])
@pytest.mark.parametrize("xt,inter,rot", [(BF16, False, 128), (F32, True, 64)])
def test_appends_of_many_waves(q4k, dtype, block, xt, inter, rot):
    """Thousands of tokens of many heads, enough for the kernel of five CTAs an SM."""
    cache = plain8.Cache([2500, 400], 2600, 128, block, 2, 128, dtype, seed=12)
    _append(q4k, cache, [2500, 310], [0, 90], H=48, rot=rot, xt=xt, interleaved=inter, seed=13)


@pytest.mark.parametrize("form", FORMS)
def test_graphs_share_scratch(q4k, form):
    """Two captured graphs and eager calls in turn, all on the library's one pool of scratch, each with lengths and values
    of its own; then both graphs at once on two streams."""
    g = torch.Generator().manual_seed(31)
    H, KH, D, page, n = 8, 2, 128, 16, 24
    sets = []
    for i, lens in enumerate(([300, 90], [1000, 24])):
        ((kc, ks, _), (vc, vs, _)), pt = _cache(g, lens, page, 16 if i else 4, KH, D, I8)
        q = torch.randn(2 * n, H, D, generator=g).bfloat16().cuda()
        args = (q, kc, vc, ks, vs, pt.cuda(), _dev([0, n, 2 * n]), _dev(lens))
        want = q4k.paged_attention8(*args, form=form)
        sets.append((args, want, torch.zeros_like(want), torch.cuda.CUDAGraph()))
    for args, want, out, graph in sets:
        with torch.cuda.graph(graph):
            q4k.paged_attention8(*args, out, form=form)
            q4k.paged_attention8(*args, out, form=form, pdl=True)
    for _ in range(3):
        for args, want, out, graph in sets:
            out.zero_()
            graph.replay()
            eager = q4k.paged_attention8(*args, form=form)
            assert torch.equal(out, want) and torch.equal(eager, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for s, (args, want, out, graph) in zip(streams, sets):
            with torch.cuda.stream(s):
                out.zero_()
                graph.replay()
        eager = [q4k.paged_attention8(*args, form=form, stream=s) for s, (args, *_) in zip(streams, sets)]
        torch.cuda.synchronize()
        for y, (_, want, out, _) in zip(eager, sets):
            assert torch.equal(out, want) and torch.equal(y, want)
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
def test_padded_batches(q4k, form):
    """Sequences of no tokens, a cached length of zero, rows behind the last sequence: those of out, lse and q_out are left
    as they were, and nothing of the others changes."""
    g = torch.Generator().manual_seed(41)
    H, KH, D, page, lens, new = 4, 2, 64, 32, [50, 0, 7, 130, 0], [20, 0, 7, 3, 0]
    ((kc, ks, _), (vc, vs, _)), pt = _cache(g, lens, page, 8, KH, D, E4M3)
    T = sum(new)
    q = torch.randn(T + 9, H, D, generator=g).bfloat16().cuda()
    index = (pt.cuda(), _dev(_starts(new)), _dev(lens))
    want = q4k.paged_attention8(q[:T], kc, vc, ks, vs, *index, form=form)
    out, lse = torch.full_like(q, 7.0), torch.full((T + 9, H), 7.0, device="cuda")
    q4k.paged_attention8(q, kc, vc, ks, vs, *index, out, lse=lse, form=form)
    assert torch.equal(out[:T], want) and bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all()) and bool((lse[:T] != 7).all())
    k = torch.randn(T + 9, KH, D, generator=g).cuda()
    tab, q_out = q4k.rope_table(200, D), torch.full_like(q, 7.0)
    a, b = ([t.clone() for t in (kc, vc, ks, vs)] for _ in range(2))
    q4k.kv_append8(k, k, *a, *index, table=tab, q=q, q_out=q_out)
    first = q4k.kv_append8(k[:T], k[:T], *b, *index, table=tab, q=q[:T])
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert all(same(x, y) for x, y in zip(a, b)) and torch.equal(q_out[:T], first) and bool((q_out[T:] == 7).all())
    r = [torch.full((T + 9, KH, D), 7.0, device="cuda") for _ in range(2)]
    q4k.kv_read8(*a, *index, T + 9, *r)
    assert all(bool((x[T:] == 7).all()) and bool((x[:T] != 7).any()) for x in r)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
def test_rows_before_the_first_sequence(q4k, form):
    """A call whose first sequence does not begin with its first row: the rows before it stay as they are."""
    g = torch.Generator().manual_seed(43)
    H, KH, D, page, lens, new, skip = 8, 2, 64, 16, [200, 77], [150, 9], 301
    ((kc, ks, _), (vc, vs, _)), pt = _cache(g, lens, page, 16, KH, D, I8)
    q = torch.randn(skip + sum(new), H, D, generator=g).bfloat16().cuda()
    start = torch.tensor(_starts(new), dtype=torch.int32).cuda()
    want = q4k.paged_attention8(q[skip:], kc, vc, ks, vs, pt.cuda(), start, _dev(lens), form=form)
    out = torch.full_like(q, 7.0)
    q4k.paged_attention8(q, kc, vc, ks, vs, pt.cuda(), start + skip, _dev(lens), out, form=form)
    # (the same tiles; which CTA holds which part of them may differ)
    assert bool((out[:skip] == 7).all())
    assert (out[skip:].double() - want.double()).abs().max() <= 2.0 ** -7 * want.double().abs().max()
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("qt", [F32, BF16])
def test_heads_of_one_memory(q4k, form, qt):
    """Cache heads that are one (a stride of 0, which TMA boxes do not take), a table row shared by two sequences."""
    H, KH, D, page, lens, new = 8, 4, 128, 32, [100, 90], [40, 3]
    if not _takes(form, qt, qt, D, page, 1.0, H // KH, 0.0):
        pytest.skip("not a form of fp32 calls")
    g = torch.Generator().manual_seed(47)
    ((kc, ks, _), (vc, vs, _)), pt = _cache(g, lens[:1], page, 4, 1, D, E4M3)
    pt = pt.expand(2, -1)
    q = torch.randn(sum(new), H, D, generator=g).to(qt).cuda()
    index = (_dev(_starts(new)), _dev(lens))
    one = [t.expand(*t.shape[:2], KH, *t.shape[3:]) for t in (kc, vc, ks, vs)]
    full = [t.contiguous() for t in one]
    want = q4k.paged_attention8(q, *full, pt.contiguous().cuda(), *index, form=form)
    got = q4k.paged_attention8(q, *one, pt.cuda(), *index, form=form)
    assert torch.equal(got, want)
    r = q4k.kv_read8(*one, pt.cuda(), *index, sum(new))
    assert all(torch.equal(x, y) for x, y in zip(r, q4k.kv_read8(*full, pt.cuda(), *index, sum(new))))
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("block", [4, 16, 64])
def test_scales_of_both_signs(q4k, form, block):
    """A cache filled by someone else may have negative scales, the largest among them."""
    H, KH, D, page, lens, new = 4, 2, 128, 64, [300, 90], [40, 3]
    for qt, ct in ((F32, I8), (BF16, E4M3), (F16, I8)):
        if not _takes(form, qt, qt, D, page, 1.0, H // KH, 0.0):
            continue
        g = torch.Generator().manual_seed(53)
        sides, pt = _cache(g, lens, page, block, KH, D, ct)
        moved = []
        for c, s, vals in sides:
            sign = torch.where(torch.rand(s.shape, generator=g) < 0.5, -1.0, 1.0)
            sign = torch.where(s.cpu() > s.cpu().nan_to_num().median(), sign * 16, sign) if s is sides[1][1] else sign
            out = []
            for b, n in enumerate(lens):
                at = torch.arange(n)
                out.append(vals[b] * sign[pt[b].long()[at // page], at % page // block].double()[..., None])
            moved.append((c, s * sign.cuda(), out))
        (kc, ks, keys), (vc, vs, vals) = moved
        q = torch.randn(sum(new), H, D, generator=g).to(qt)
        y = q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, pt.cuda(), _dev(_starts(new)), _dev(lens), form=form)
        ref, _, bound, _ = _bound(q, keys, vals, dict(new=new, len=lens), 1 / math.sqrt(D), qt, qt != F32 and form in (None, "many"),
                                  vs.abs(), vc)
        assert ((y.double().cpu() - ref).abs() <= bound).all()
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("ct", [I8, E4M3])
def test_append_to_a_negative_scale(q4k, ct):
    """The older tokens of a block keep their values under the new, positive scale."""
    past, n, KH, D, page, block = 5, 3, 2, 64, 16, 16
    g = torch.Generator().manual_seed(57)
    for old in (-0.5, -1e-4):
        cache = plain8.Cache([past + n], past + n, page, block, KH, D, ct, seed=8)
        for s in cache.scales:
            s[:] = old
        dev = cache.device()
        v = torch.randn(n, KH, D, generator=g)
        q4k.kv_append8(v.cuda(), v.cuda(), *dev[:4], dev[4], _dev([0, n]), _dev([past + n]))
        after = copy.copy(cache)
        after.codes, after.scales = [t.cpu() for t in dev[:2]], [t.cpu() for t in dev[2:4]]
        for side in (0, 1):
            got = after.scales[side][cache.table[0, 0].long(), 0].double()
            want = torch.maximum(v.double().abs().amax((0, 2)) / plain8.TOP[ct], torch.tensor(-old).double())
            assert ((got - want).abs() <= 2.0 ** -23 * want).all()
            y = cache.values(side, 0, torch.arange(past)) / got[:, None]
            near = plain8.half_step(y * (1 + 2.0 ** -20), ct) * (1 + 2.0 ** -20) + y.abs() * 2.0 ** -22
            assert ((after.values(side, 0, torch.arange(past)) / got[:, None] - y).abs() <= near).all()
            y = v.double() / got[:, None]
            near = plain8.half_step(y * (1 + 2.0 ** -20), ct) * (1 + 2.0 ** -20) + y.abs() * 2.0 ** -22
            assert ((after.values(side, 0, torch.arange(past, past + n)) / got[:, None] - y).abs() <= near).all()
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
def test_old_contents_of_pages(q4k, form):
    """What earlier sequences left in a page's later slots, large scales among it, changes nothing."""
    g = torch.Generator().manual_seed(51)
    H, KH, D, page, block, lens, new = 4, 2, 128, 128, 2, [131, 40], [37, 5]
    ((kc, ks, _), (vc, vs, _)), pt = _cache(g, lens, page, block, KH, D, I8)
    q = torch.randn(sum(new), H, D, generator=g).bfloat16().cuda()
    index = (pt.cuda(), _dev(_starts(new)), _dev(lens))
    want = q4k.paged_attention8(q, kc, vc, ks, vs, *index, form=form)
    for t in (kc, vc):
        t[t == -128] = 127
    for t in (ks, vs):
        t[torch.isnan(t)] = 1e30
    assert torch.equal(q4k.paged_attention8(q, kc, vc, ks, vs, *index, form=form), want)
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("qt,block,first", [(BF16, 16, False), (F16, 4, True)])
def test_passes_of_heads(q4k, qt, block, first):
    """A page table of a million positions: the widened keys and values of 6 heads take 6.6 GB, so they go in passes."""
    g = torch.Generator().manual_seed(61)
    H, KH, D, page, lens, new = 12, 6, 128, 128, [700, 90], [150, 33]
    ((kc, ks, keys), (vc, vs, vals)), pt = _cache(g, lens, page, block, KH, D, I8, first)
    wide = torch.full((2, 8500), -1, dtype=torch.int32)
    wide[:, :pt.shape[1]] = pt
    q = torch.randn(sum(new), H, D, generator=g).to(qt)
    slopes = torch.tensor([2.0 ** (-0.5 * i - 1) for i in range(H)])
    lse = torch.zeros(sum(new), H, device="cuda")
    call = lambda **kw: q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, wide.cuda(), _dev(_starts(new)), _dev(lens), slopes=slopes.cuda(),
                                             lse=lse, form="many", **kw)
    y = call()
    ref, rl, bound, off = _bound(q, keys, vals, dict(new=new, len=lens), 1 / math.sqrt(D), qt, True, vs, vc, slopes)
    assert ((y.double().cpu() - ref).abs() <= bound).all()
    assert ((lse.double().cpu() - rl).abs() <= 2.0 ** -12 + 2.0 ** -20 * rl.abs() + off).all()
    for _ in range(3):
        assert torch.equal(call(pdl=True), y)
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(y)
    args = (q.cuda(), kc, vc, ks, vs, wide.cuda(), _dev(_starts(new)), _dev(lens), out)
    bias = slopes.cuda()
    with torch.cuda.graph(graph):
        q4k.paged_attention8(*args, slopes=bias, form="many")
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, y)
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("ct,qt,mask", [(I8, BF16, {}), (E4M3, F16, dict(window=60)), (I8, BF16, dict(prefix=[30, 200, 0, 90, 5])),
                                        (E4M3, BF16, dict(kv_start=True))])
def test_passes_of_sequences(q4k, ct, qt, mask):
    """A page table of three million positions: two sequences of a head a pass, five sequences, three of them with no new tokens
    at an end or between."""
    g = torch.Generator().manual_seed(63)
    H, KH, D, page, lens, new = 4, 2, 128, 64, [300, 40, 129, 700, 90], [0, 40, 0, 133, 260]
    lens[4] = 260
    ((kc, ks, keys), (vc, vs, vals)), pt = _cache(g, lens, page, 4, KH, D, ct)
    wide = torch.full((5, 3 * 2 ** 20 // page), -1, dtype=torch.int32)
    wide[:, :pt.shape[1]] = pt
    case = dict(new=new, len=lens, **mask)
    if mask.get("kv_start"):
        case["kv_start"] = [(n - m + i) // 50 * 50 for n, m in zip(lens, new) for i in range(m)]
    q = torch.randn(sum(new), H, D, generator=g).to(qt)
    lse = torch.zeros(sum(new), H, device="cuda")
    kw = dict(window=mask.get("window", 0), prefix_len=None if "prefix" not in mask else _dev(mask["prefix"]),
              kv_start=None if "kv_start" not in mask else _dev(case["kv_start"]))
    call = lambda **more: q4k.paged_attention8(q.cuda(), kc, vc, ks, vs, wide.cuda(), _dev(_starts(new)), _dev(lens), lse=lse,
                                               form="many", **kw, **more)
    y = call()
    ref, rl, bound, off = _bound(q, keys, vals, case, 1 / math.sqrt(D), qt, True, vs, vc)
    assert ((y.double().cpu() - ref).abs() <= bound).all()
    assert ((lse.double().cpu() - rl).abs() <= 2.0 ** -12 + 2.0 ** -20 * rl.abs() + off).all()
    for _ in range(3):
        assert torch.equal(call(pdl=True), y)
    assert q4k.device_error_flags() == 0


def test_no_room_for_a_head(q4k):
    """Past 4 GiB for one head of a sequence the widened form is refused by name and not chosen by itself."""
    g = torch.Generator().manual_seed(71)
    H, KH, D, page, lens, new = 4, 2, 64, 16, [400], [300]
    ((kc, ks, keys), (vc, vs, vals)), pt = _cache(g, lens, page, 16, KH, D, I8)
    wide = torch.full((1, 2 ** 24 // page + 1), -1, dtype=torch.int32)
    wide[:, :pt.shape[1]] = pt
    q = torch.randn(300, H, D, generator=g).bfloat16()
    args = (q.cuda(), kc, vc, ks, vs, wide.cuda(), _dev([0, 300]), _dev(lens))
    with pytest.raises(q4k.Q4KError) as e:
        q4k.paged_attention8(*args, form="many")
    assert e.value.status == 1
    y = q4k.paged_attention8(*args)
    ref, _, bound, _ = _bound(q, keys, vals, dict(new=new, len=lens), 0.125, BF16, False, vs, vc)
    assert ((y.double().cpu() - ref).abs() <= bound).all()
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("form", FORMS)
def test_every_byte_as_a_code(q4k, form):
    """All 256 codes (but NaN) of both types as keys and as values, at positions of every residue."""
    for ct in (I8, E4M3):
        codes = torch.arange(256, dtype=torch.uint8)
        if ct == E4M3:
            codes = codes[(codes & 0x7F) != 0x7F]
        n, D, page, block = len(codes) + 1, 64, 16, 16
        pages = -(-n // page)
        kc = torch.zeros(pages, page, 1, D, dtype=torch.uint8)
        flat = kc.view(-1, D)
        for d in range(D):     # each column in another order
            flat[:len(codes), d] = codes.roll(7 * d)
        vc = kc.flip(-1).contiguous()
        s = torch.full((pages, 1, 1), 2.0 ** -9)
        q = torch.zeros(1, 2, D)
        q[0, 0, 3], q[0, 1] = 1.0, 0.125
        val = lambda c: c.view(ct).view(-1, 1, D)[:n].float().double() * 2.0 ** -9
        for qt in (F32, BF16):
            if not _takes(form, qt, qt, D, page, 1.0, 2, 0.0):
                continue
            y = q4k.paged_attention8(q.to(qt).cuda(), kc.view(ct).cuda(), vc.view(ct).cuda(), s.cuda(), s.cuda(),
                                     torch.arange(pages, dtype=torch.int32).view(1, -1).cuda(), _dev([0, 1]), _dev([n]), scale=1.0, form=form)
            ref, _, bound, _ = _bound(q, [val(kc)], [val(vc)], dict(new=[1], len=[n]), 1.0, qt, qt == BF16 and form in (None, "many"), s,
                                      vc.view(ct))
            assert ((y.double().cpu() - ref).abs() <= bound).all()
    assert q4k.device_error_flags() == 0
