"""CPU-side checks of the 8-bit cache's entry points: the packed structures match the header, argument errors come back
before any device call, the host side launches what it should (over a runtime that runs nothing), and the Python calls
take tensors of one device and give outputs of their stream."""
import math
import os
import shutil
import struct
import subprocess

import pytest

torch = pytest.importorskip("torch")
from fake_runtime import fake, fake_path   # noqa: F401,E402
from test_attention_abi import BAD_CACHES, OK, _attention   # noqa: E402
from test_attention_binding import Tensor, World   # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# The structures of include/q4k.h, field by field (native alignment).
CACHE8 = struct.Struct("@2P 6q 4q P 2q 2P 2q 2i 2P 6q q")
HEADS = "3P 6q 2i"
NORM = struct.Struct(f"@{HEADS} {HEADS} 2P 4q f 3i")
APPEND8 = struct.Struct("@4P 8q 2P 3q 6i 2P 2q f i")
READ8 = struct.Struct("@2P 4q 2i")
F32, BF16, I32, I8 = torch.float32, torch.bfloat16, torch.int32, torch.int8


@pytest.fixture(scope="module")
def L():
    from q4_dequant_gemv_gb300 import _build
    _build.build()
    import q4_dequant_gemv_gb300 as m
    return m.lib()


def test_structures_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "q4k.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu ", sizeof(q4k_paged_cache8), sizeof(q4k_norm_rope_args), sizeof(q4k_append8_args), '
                   'sizeof(q4k_read8_args));\n'
                   'printf("%zu %zu %zu %zu\\n", offsetof(q4k_paged_cache8, block), offsetof(q4k_norm_rope_args, eps), '
                   'offsetof(q4k_append8_args, eps), offsetof(q4k_read8_args, type));\nreturn 0; }\n')
    exe = str(tmp_path / "s")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    structs = [CACHE8, NORM, APPEND8, READ8]
    assert got[:4] == [s.size for s in structs]
    assert got[4:] == [CACHE8.size - 8, NORM.size - 16, APPEND8.size - 8, READ8.size - 8]


def _cache8(**kw):
    d = dict(k=OK, v=OK, kp=2048, ks=128, kh=64, vp=2048, vs=128, vh=64, pages=4, size=16, heads=2, dim=64, table=OK, row=2,
             most=2, start=OK, len=OK, batch=1, tokens=2, type=3, pad=0, k_scale=OK, v_scale=OK, ksp=8, ksb=2, ksh=1, vsp=8,
             vsb=2, vsh=1, block=4) | kw
    return CACHE8.pack(*d.values())


def _norm(**kw):
    d = dict(x=OK, y=OK, w=OK, heads=3, xt=192, xh=64, yt=192, yh=64, wh=0, xc=0, yc=0,
             x2=OK, y2=OK, w2=OK, heads2=1, xt2=64, xh2=64, yt2=64, yh2=64, wh2=0, xc2=0, yc2=0,
             pos=OK, table=OK, tokens=2, dim=64, rot=64, rows=8, eps=1e-6, inter=0, flags=0, pad=0) | kw
    return NORM.pack(*d.values())


def _append8(**kw):
    d = dict(k=OK, v=OK, q=0, qo=0, kt=128, kh=64, vt=128, vh=64, qt=0, qh=0, ot=0, oh=0, pos=0, table=OK, rows=8, rot=64,
             heads=0, kc=0, qc=0, oc=0, inter=0, flags=0, pad=0, qw=0, kw=0, qwh=0, kwh=0, eps=1e-6, pad2=0) | kw
    return APPEND8.pack(*d.values())


def _read8(**kw):
    d = dict(k=OK, v=OK, kt=128, kh=64, vt=128, vh=64, type=2, flags=0) | kw
    return READ8.pack(*d.values())


BAD_CACHES8 = tuple(b for b in BAD_CACHES if b != dict(type=0)) + (
    dict(type=0), dict(type=1), dict(type=5), dict(block=0), dict(block=3), dict(block=32), dict(block=-4), dict(size=48, block=32),
    dict(size=512, block=256), dict(k_scale=0), dict(v_scale=0), dict(dim=60), dict(dim=264))


def test_norm_rope_arguments(L):
    f = L.q4k_norm_rope
    for bad in (dict(x=0), dict(y=0), dict(x2=0), dict(y2=0), dict(heads=0), dict(heads2=0), dict(xc=3), dict(yc2=-1), dict(tokens=-1),
                dict(dim=60), dict(dim=0), dict(dim=264), dict(rot=63), dict(rot=66), dict(rot=-2), dict(rows=-1), dict(pos=0),
                dict(table=0), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(inter=2), dict(flags=2)):
        assert f(_norm(**bad), 0) == 1, bad
    for bad in (dict(x=OK + 2), dict(y2=OK + 1, yc2=1), dict(w=OK + 2), dict(w2=OK + 1), dict(pos=OK + 2), dict(table=OK + 1)):
        assert f(_norm(**bad), 0) == 2, bad
    assert f(None, 0) == 1
    for ok in (dict(tokens=0, x=0, y=0, pos=0, table=0, x2=0, y2=0), dict(x2=0, y2=0), dict(rot=0, pos=0, table=0), dict(w=0, w2=0)):
        assert f(_norm(**ok), 0) in (0, 3, 4)


def test_append_and_read_arguments(L):
    for bad in BAD_CACHES8:
        assert L.q4k_kv_append8(_cache8(**bad), _append8(), 0) == 1, bad
        assert L.q4k_kv_read8(_cache8(**bad), _read8(), 0) == 1, bad
    for bad in (dict(k=0), dict(v=0), dict(table=0), dict(rows=-1), dict(rot=1), dict(rot=66), dict(kc=3), dict(inter=3), dict(q=OK),
                dict(qo=OK), dict(q=OK, qo=OK, heads=0), dict(q=OK, qo=OK, heads=2, qc=9), dict(flags=8), dict(eps=-1.0),
                dict(eps=math.nan)):
        assert L.q4k_kv_append8(_cache8(), _append8(**bad), 0) == 1, bad
    for bad in (dict(k=OK + 2), dict(pos=OK + 1), dict(kw=OK + 2), dict(qw=OK + 1)):
        assert L.q4k_kv_append8(_cache8(), _append8(**bad), 0) == 2, bad
    for bad in (dict(type=3), dict(type=-1), dict(flags=2)):
        assert L.q4k_kv_read8(_cache8(), _read8(**bad), 0) == 1, bad
    assert L.q4k_kv_read8(_cache8(), _read8(k=OK + 1), 0) == 2
    for bad in (dict(k_scale=OK + 2), dict(v_scale=OK + 1), dict(start=OK + 2)):
        assert L.q4k_kv_append8(_cache8(**bad), _append8(), 0) == 2, bad
    for f, a in ((L.q4k_kv_append8, _append8()), (L.q4k_kv_read8, _read8())):
        assert f(None, a, 0) == 1 and f(_cache8(), None, 0) == 1
        assert f(_cache8(tokens=0), a, 0) in (0, 3, 4) and f(_cache8(k=OK + 1, ks=129), a, 0) in (0, 3, 4)


def test_attention_arguments(L):
    f = L.q4k_paged_attention8
    for bad in BAD_CACHES8 + (dict(dim=72), dict(dim=8)):
        assert f(_cache8(**bad), _attention(), 0) == 1, bad
    for bad in (dict(q=0), dict(out=0), dict(heads=0), dict(heads=3), dict(window=-1), dict(scale=math.nan), dict(cap=-1.0), dict(qc=3),
                dict(oc=7), dict(causal=2), dict(flags=2)):
        assert f(_cache8(), _attention(**bad), 0) == 1, bad
    for bad in (dict(k=OK + 8), dict(kp=2056), dict(vs=136), dict(vh=8), dict(k_scale=OK + 2)):
        assert f(_cache8(**bad), _attention(), 0) == 2, bad
    for bad in (dict(q=OK + 4), dict(out=OK + 8), dict(qt=257), dict(lse=OK + 2)):
        assert f(_cache8(), _attention(**bad), 0) == 2, bad
    assert f(None, _attention(), 0) == 1 and f(_cache8(), None, 0) == 1
    assert f(_cache8(tokens=0), _attention(q=0, out=0), 0) in (0, 3, 4)
    # the 16-bit calls do not take codes
    from test_attention_abi import _cache
    assert L.q4k_paged_attention(_cache(type=3), _attention(), 0) == 1 and L.q4k_paged_attention(_cache(type=4), _attention(), 0) == 1


def test_no_device_reports_status(L):
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert L.q4k_norm_rope(_norm(), 0) in (3, 4)
    assert L.q4k_kv_append8(_cache8(), _append8(), 0) in (3, 4)
    assert L.q4k_kv_read8(_cache8(), _read8(), 0) in (3, 4)
    assert L.q4k_paged_attention8(_cache8(), _attention(), 0) in (3, 4)


# ---------------------------------------------------------------- the host side

def _bind(lib):
    import ctypes
    P, S = ctypes.c_void_p, ctypes.c_char_p
    lib.L.q4k_norm_rope.argtypes = [S, P]
    lib.L.q4k_kv_append8.argtypes = lib.L.q4k_kv_read8.argtypes = lib.L.q4k_paged_attention8.argtypes = [S, S, P]
    return lib.L


FORMS = {"cluster8": 1, "cluster16": 2, "cluster32": 3, "split8": 4, "split16": 5, "split32": 6, "many": 7}


@pytest.mark.parametrize("form", FORMS)
def test_every_device_gets_what_it_needs(fake, form):   # noqa: F811
    L = _bind(fake)
    for d in (0, 1, 0, 3, 1):
        fake.device(d)
        assert L.q4k_paged_attention8(_cache8(), _attention(flags=FORMS[form] << 8), 0) == 0, f"device {d}"
        got = fake.launches()
        assert all(x.device == d for x in got)
        assert (b"widen" in got[0].kernel) == (form == "many") and len(got) == {"c": 1, "s": 2, "m": 3}[form[0]]
        assert fake.blocks(d) == 0


@pytest.mark.parametrize("form", ["cluster8", "split8", "many"])
@pytest.mark.parametrize("skip", [0, 1, 2])
@pytest.mark.parametrize("name", ["cudaFuncSetAttribute", "cudaMemPoolCreate", "cudaMallocFromPoolAsync", "cudaLaunchKernelExC"])
def test_a_failure_is_not_kept(fake, form, name, skip):   # noqa: F811
    """The call that meets it says so and leaves no scratch behind; the next one works."""
    L = _bind(fake)
    fake.fail(name, skip=skip)
    first = L.q4k_paged_attention8(_cache8(), _attention(flags=FORMS[form] << 8), 0)
    assert first in (0, 4) and fake.blocks(0) == 0
    if first == 0:      # the call does not get that far
        assert skip > 0 or (form == "cluster8" and "Pool" in name)
    fake.fail(name, 0)
    fake.launches()
    assert L.q4k_paged_attention8(_cache8(), _attention(flags=FORMS[form] << 8), 0) == 0
    assert fake.launches() and fake.blocks(0) == 0


def test_passes_of_heads(fake):   # noqa: F811
    """A widened cache past 4 GiB goes through in passes of as many heads as fit, then of sequences, one past it for a head of
    a sequence not at all."""
    L = _bind(fake)
    def call(heads, most, form=7, batch=1, tokens=2):
        c = _cache8(size=128, heads=heads, dim=128, block=16, kh=128, ks=128 * heads, kp=128 * 128 * heads, vh=128, vs=128 * heads,
                    vp=128 * 128 * heads, pages=1 << 20, row=most, most=most, batch=batch, tokens=tokens)
        return L.q4k_paged_attention8(c, _attention(heads=heads, qt=128 * heads, qh=128, ot=128 * heads, oh=128, flags=form << 8), 0)
    for heads, most, batch, passes in ((8, 1024, 1, 1),       # 131072 positions of 8 heads: 0.5 GiB
                                       (8, 1024, 16, 3),      # 8 GiB and a little more
                                       (3, 16384, 1, 1), (3, 16384, 2, 3),      # a head 2 GiB
                                       (2, 30000, 5, 6),      # a sequence 1.8: two a pass
                                       (1, 8, 70000, 9)):     # 512 KiB a sequence
        assert call(heads, most, batch=batch) == 0
        got = fake.launches()
        assert [b"widen" in x.kernel for x in got].count(True) == passes and len(got) == 3 * passes, (heads, most, batch)
        assert fake.blocks(0) == 0
    assert call(1, 1 << 16) == 1       # 8 million positions of a head: 4 GiB and the factors
    assert call(1, 1 << 16, form=0) == 0 and not any(b"widen" in x.kernel for x in fake.launches())


def test_less_memory_makes_smaller_passes(fake):   # noqa: F811
    """An allocation that fails is tried again with half the heads, then half the sequences; small ones are not."""
    L = _bind(fake)
    def call(heads, most, batch):
        c = _cache8(size=128, heads=heads, dim=128, block=16, kh=128, ks=128 * heads, kp=128 * 128 * heads, vh=128, vs=128 * heads,
                    vp=128 * 128 * heads, pages=1 << 20, row=most, most=most, batch=batch)
        return L.q4k_paged_attention8(c, _attention(heads=heads, qt=128 * heads, qh=128, ot=128 * heads, oh=128, flags=7 << 8), 0)
    passes = lambda: [b"widen" in x.kernel for x in fake.launches()].count(True)
    for times, want in ((0, 1), (1, 2), (2, 4), (3, 8), (4, 16)):   # 8 heads of 2 sequences, 64 MiB each
        fake.fail("cudaMallocFromPoolAsync", times)
        assert call(8, 1024, 2) == 0 and passes() == want and fake.blocks(0) == 0, times
    fake.fail("cudaMallocFromPoolAsync", 5)
    assert call(8, 1024, 2) == 4 and passes() == 0 and fake.blocks(0) == 0
    fake.fail("cudaMallocFromPoolAsync", 1)
    assert call(8, 8, 2) == 4 and passes() == 0
    fake.fail("cudaMallocFromPoolAsync", 0)
    assert call(8, 8, 2) == 0 and passes() == 1


def test_wide_and_narrow_rows(fake):   # noqa: F811
    """Aligned rows of sizes that fit take the wide kernels; strides that no index uses make no difference."""
    L = _bind(fake)
    wide = lambda: [b"Lb1" in x.kernel for x in fake.launches()]   # the kernels' first template argument
    for kw, want in ((dict(), True), (dict(tokens=1, xt=1, yt=-7, xt2=3), True), (dict(heads=1, xh=3, yh=5, wh=7, xt=64, yt=64), True),
                     (dict(xt=193), False), (dict(yh2=66, heads2=2), False), (dict(rot=20), False), (dict(w=OK + 4), False),
                     (dict(w2=OK + 4), False), (dict(wh=66), False), (dict(wh=68), True)):
        assert L.q4k_norm_rope(_norm(**kw), 0) == 0
        assert wide() == [want], kw
    for cache, kw, want in ((dict(), {}, True), (dict(pages=1, kp=2051, vp=1, ksp=9), {}, True), (dict(size=4, ksb=77), {}, True),
                            (dict(ks=129), {}, False), (dict(k=OK + 4), {}, False), (dict(), dict(kw=OK + 4), False),
                            (dict(), dict(kt=129), False)):
        assert L.q4k_kv_append8(_cache8(**cache), _append8(**kw), 0) == 0
        assert wide() == [want], (cache, kw)
    for cache, kw, want in ((dict(), {}, True), (dict(vs=129), {}, False), (dict(), dict(vt=129), False)):
        assert L.q4k_kv_read8(_cache8(**cache), _read8(**kw), 0) == 0
        assert wide() == [want], (cache, kw)


# ---------------------------------------------------------------- the Python calls

class World8(World):
    def __init__(self, monkeypatch):
        super().__init__(monkeypatch)
        import ctypes
        import types
        from q4_dequant_gemv_gb300 import _cache8
        _cache8._calls = None
        two, three = (ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * n) for n in (2, 3))
        note = lambda name: lambda *a: self.calls.append((name, a[-1] or 0)) or 0
        for name, proto in (("norm_rope", two), ("kv_append8", three), ("kv_read8", three), ("paged_attention8", three)):
            setattr(self.lib, "q4k_" + name, proto(note(name)))
        monkeypatch.setattr(_cache8, "torch", types.SimpleNamespace(int8=I8, float8_e4m3fn=torch.float8_e4m3fn, bfloat16=BF16))
        self.m8 = _cache8

    def cache8(self, device=0):
        return [Tensor((3, 16, 2, 64), I8, device) for _ in range(2)] + [Tensor((3, 4, 2), F32, device) for _ in range(2)]


@pytest.fixture
def world(monkeypatch):
    yield World8(monkeypatch)
    import q4_dequant_gemv_gb300._attention as m
    import q4_dequant_gemv_gb300._cache8 as m8
    m._calls = m8._calls = None


def _calls(w, d=0, **kw):
    x = lambda h=2: Tensor((4, h, 64), device=d)
    return {
        "norm_rope": ([x(4), x(), Tensor((4,), I32, d), Tensor((8, 64), F32, d), Tensor((64,), F32, d), Tensor((2, 64), F32, d)],
                      lambda *a, **k: w.m8.norm_rope(*a, **kw, **k)),
        "kv_append8": ([x(), x(), *w.cache8(d), *w.index(d)], lambda *a, **k: w.m8.kv_append8(*a, q=x(4), q_weight=Tensor((64,), F32, d), **kw, **k)),
        "kv_read8": ([*w.cache8(d), *w.index(d)], lambda *a, **k: w.m8.kv_read8(*a, 4, **kw, **k)),
        "paged_attention8": ([x(4), *w.cache8(d), *w.index(d)], lambda *a, **k: w.m8.paged_attention8(*a, **kw, **k)),
    }


def test_outputs_are_the_calls_streams_own(world):
    for name, (args, f) in _calls(world, stream=world.side).items():
        world.calls.clear()
        out = f(*args)
        for y in out if isinstance(out, tuple) else (out,):
            assert y.allocated_on is world.side and world.main in y.recorded, name
        assert world.calls == [(name, 77)] and world.now is world.main, name
    for name, (args, f) in _calls(world).items():
        world.calls.clear()
        out = f(*args)
        for y in out if isinstance(out, tuple) else (out,):
            assert y.allocated_on is world.main and not y.recorded, name
        assert world.calls == [(name, 0)], name


def test_tensors_of_several_devices_are_refused(world):
    """Every tensor argument by itself, and all of them where the device is not current."""
    for name, (args, f) in _calls(world).items():
        other = _calls(world, 1)[name][0]
        for i in range(len(args)):
            world.calls.clear()
            with pytest.raises(ValueError, match="cuda:"):
                f(*args[:i], other[i], *args[i + 1:])
            assert not world.calls, (name, i)
        with pytest.raises(ValueError, match="cuda:"):
            f(*other)
    for name, (args, f) in _calls(world, 1).items():
        world.device = 1
        world.calls.clear()
        f(*args)
        assert len(world.calls) == 1


def test_bad_tensors_are_refused(world):
    w = world
    args, f = _calls(w)["norm_rope"]
    for i, bad in ((0, Tensor((4, 4, 64), torch.float64)), (1, Tensor((3, 2, 64))), (1, Tensor((4, 2, 32))), (2, Tensor((3,), I32)),
                   (3, Tensor((8, 66))), (3, Tensor((8, 63))), (4, Tensor((32,))), (4, Tensor((3, 64))), (4, Tensor((64,), BF16)),
                   (5, Tensor((2, 64), strides=(128, 2)))):
        with pytest.raises((ValueError, TypeError)):
            f(*args[:i], bad, *args[i + 1:])
    for kw in (dict(eps=-1.0), dict(eps=math.inf), dict(k_out=Tensor((4, 3, 64))), dict(out_dtype=torch.int8)):
        with pytest.raises((ValueError, TypeError)):
            f(*args, **kw)
    with pytest.raises(ValueError):
        w.m8.norm_rope(args[0], None, *args[2:])       # k_weight without k
    with pytest.raises(ValueError):
        w.m8.norm_rope(args[0], table=args[3])         # no pos
    args, f = _calls(w)["kv_append8"]
    for i, bad in ((2, Tensor((3, 16, 2, 64), BF16)), (3, Tensor((3, 16, 2, 64), torch.float8_e4m3fn)), (4, Tensor((3, 4, 2), BF16)),
                   (4, Tensor((3, 3, 2))), (5, Tensor((3, 2, 2))), (5, Tensor((3, 4))), (0, Tensor((4, 3, 64))), (6, Tensor((1, 2), torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            f(*args[:i], bad, *args[i + 1:])
    with pytest.raises(ValueError):
        w.m8.kv_append8(*args, q_weight=Tensor((64,)))  # no q
    args, f = _calls(w)["kv_read8"]
    for kw in (dict(k=Tensor((5, 2, 64), BF16)), dict(k=Tensor((4, 2, 64), BF16), v=Tensor((4, 2, 64), F32)), dict(dtype=torch.int8)):
        with pytest.raises((ValueError, TypeError)):
            f(*args, **kw)
    with pytest.raises((ValueError, OverflowError)):
        w.m8.kv_read8(*args, -1)
    assert not w.calls
