"""CPU-side checks of the rotary, append and attention entry points: the packed structures match the header, and
argument errors come back before any device call."""
import ctypes
import math
import os
import shutil
import struct
import subprocess

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# The structures of include/q4k.h, field by field (native alignment).
ROPE = struct.Struct("@4P 5q 4q 4i")
SCALE = struct.Struct("@6d 2i")
CACHE = struct.Struct("@2P 6q 4q P 2q 2P 2q 2i")
APPEND = struct.Struct("@4P 8q 2P 3q 6i")
ATTENTION = struct.Struct("@3P 4q 2q 3P 2f 6i")
OK = 0x10000   # an aligned address that is never followed on these paths


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
                   'printf("%zu %zu %zu %zu %zu ", sizeof(q4k_rope_args), sizeof(q4k_rope_scaling), '
                   'sizeof(q4k_paged_cache), sizeof(q4k_append_args), sizeof(q4k_attention_args));\n'
                   'printf("%zu %zu %zu %zu %zu\\n", offsetof(q4k_rope_args, x_type), offsetof(q4k_rope_scaling, scaling), '
                   'offsetof(q4k_paged_cache, type), offsetof(q4k_append_args, kv_type), '
                   'offsetof(q4k_attention_args, q_type));\nreturn 0; }\n')
    exe = str(tmp_path / "s")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    structs = [ROPE, SCALE, CACHE, APPEND, ATTENTION]
    assert got[:5] == [s.size for s in structs]
    ints = [4, 2, 2, 6, 6]          # the 4-byte fields at the end (the attention's follow two floats)
    assert got[5:] == [s.size - 4 * n for s, n in zip(structs, ints)]


def _scaling(base=10000.0, factor=1.0, orig=0.0, low=1.0, high=32.0, mag=1.0, kind=0):
    return SCALE.pack(base, factor, orig, low, high, mag, kind, 0)


def test_rope_table_arguments(L):
    f = L.q4k_rope_table
    assert f(OK, 4, 3, _scaling(), 0) == 1
    assert f(OK, 4, 0, _scaling(), 0) == 1
    assert f(OK, 4, 514, _scaling(), 0) == 1
    assert f(OK, -1, 64, _scaling(), 0) == 1
    assert f(0, 4, 64, _scaling(), 0) == 1
    assert f(OK, 4, 64, None, 0) == 1
    for bad in (dict(base=0.0), dict(base=math.inf), dict(factor=-1.0), dict(mag=math.nan), dict(kind=5), dict(kind=-1),
                dict(kind=3), dict(kind=4, orig=8192.0, low=4.0, high=1.0), dict(kind=3, orig=8192.0, low=0.0),
                dict(kind=3, orig=8192.0, base=1.0)):
        assert f(OK, 4, 64, _scaling(**bad), 0) == 1, bad
    assert f(OK, 4, 2, _scaling(kind=2, factor=2.0), 0) == 1     # rot / (rot - 2)
    assert f(OK + 2, 4, 64, _scaling(), 0) == 2


def _rope(**kw):
    d = dict(x=OK, y=OK, pos=OK, table=OK, tokens=2, heads=3, dim=64, rot=64, rows=8, xt=192, xh=64, yt=192, yh=64, xc=0,
             yc=0, inter=0, flags=0) | kw
    return ROPE.pack(*d.values())


def test_rope_arguments(L):
    f = L.q4k_rope
    for bad in (dict(x=0), dict(y=0), dict(pos=0), dict(table=0), dict(tokens=-1), dict(heads=0), dict(dim=0), dict(rot=63),
                dict(rot=66), dict(rot=-2), dict(rows=-1), dict(xc=3), dict(yc=-1), dict(inter=2), dict(flags=2)):
        assert f(_rope(**bad), 0) == 1, bad
    for bad in (dict(x=OK + 2), dict(y=OK + 1, yc=1), dict(pos=OK + 2), dict(table=OK + 1)):
        assert f(_rope(**bad), 0) == 2, bad
    assert f(None, 0) == 1
    assert f(_rope(tokens=0, x=0, y=0, pos=0, table=0), 0) in (0, 3, 4)


def _cache(**kw):
    d = dict(k=OK, v=OK, kp=2048, ks=128, kh=64, vp=2048, vs=128, vh=64, pages=4, size=16, heads=2, dim=64, table=OK, row=2,
             most=2, start=OK, len=OK, batch=1, tokens=2, type=2, pad=0) | kw
    return CACHE.pack(*d.values())


def _append(**kw):
    d = dict(k=OK, v=OK, q=0, qo=0, kt=128, kh=64, vt=128, vh=64, qt=0, qh=0, ot=0, oh=0, pos=0, table=OK, rows=8, rot=64,
             heads=0, kc=0, qc=0, oc=0, inter=0, flags=0, pad=0) | kw
    return APPEND.pack(*d.values())


BAD_CACHES = (dict(batch=-1), dict(tokens=-1), dict(pages=-1), dict(size=0), dict(heads=0), dict(dim=0), dict(most=-1),
              dict(row=-1), dict(type=0), dict(k=0), dict(v=0), dict(table=0), dict(start=0), dict(len=0))


def test_append_arguments(L):
    f = L.q4k_kv_append
    for bad in BAD_CACHES:
        assert f(_cache(**bad), _append(), 0) == 1, bad
    for bad in (dict(k=0), dict(v=0), dict(table=0), dict(rows=-1), dict(rot=1), dict(rot=66), dict(kc=4), dict(inter=3),
                dict(q=OK), dict(qo=OK), dict(q=OK, qo=OK, heads=0), dict(q=OK, qo=OK, heads=2, qc=9), dict(flags=8)):
        assert f(_cache(), _append(**bad), 0) == 1, bad
    assert f(_cache(k=OK + 1), _append(), 0) == 2
    assert f(_cache(start=OK + 2), _append(), 0) == 2
    assert f(_cache(), _append(v=OK + 2), 0) == 2
    assert f(None, _append(), 0) == 1 and f(_cache(), None, 0) == 1
    assert f(_cache(tokens=0), _append(k=0, v=0, table=0), 0) in (0, 3, 4)


def _attention(**kw):
    d = dict(q=OK, out=OK, lse=0, qt=256, qh=64, ot=256, oh=64, heads=4, window=0, slopes=0, prefix=0, start=0, scale=0.125,
             cap=0.0, qc=2, oc=2, causal=1, flags=0, limit=0, pad=0) | kw
    return ATTENTION.pack(*d.values())


def test_attention_arguments(L):
    f = L.q4k_paged_attention
    for bad in BAD_CACHES + (dict(dim=60), dict(dim=264)):
        assert f(_cache(**bad), _attention(), 0) == 1, bad
    for bad in (dict(q=0), dict(out=0), dict(heads=0), dict(heads=3), dict(window=-1), dict(scale=math.nan),
                dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.nan), dict(qc=3), dict(oc=7), dict(causal=2),
                dict(flags=2), dict(flags=16)):
        assert f(_cache(), _attention(**bad), 0) == 1, bad
    assert f(_cache(tokens=2 ** 30), _attention(), 0) == 1           # tokens * heads past 2^31
    for bad in (dict(k=OK + 8), dict(kp=2052), dict(vs=129), dict(vh=4)):
        assert f(_cache(**bad), _attention(), 0) == 2, bad
    for bad in (dict(q=OK + 4), dict(out=OK + 8), dict(qt=257), dict(oh=12), dict(qt=258, qc=0), dict(lse=OK + 2),
                dict(slopes=OK + 1)):
        assert f(_cache(), _attention(**bad), 0) == 2, bad
    assert f(None, _attention(), 0) == 1 and f(_cache(), None, 0) == 1
    assert f(_cache(tokens=0), _attention(q=0, out=0), 0) in (0, 3, 4)
    assert f(_cache(batch=0), _attention(q=0, out=0), 0) in (0, 3, 4)


def test_no_device_reports_status(L):
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert L.q4k_rope(_rope(), 0) in (3, 4)
    assert L.q4k_kv_append(_cache(), _append(), 0) in (3, 4)
    assert L.q4k_paged_attention(_cache(), _attention(), 0) in (3, 4)


def test_binding_refuses_host_tensors():
    import q4_dequant_gemv_gb300 as q4k
    x = torch.zeros(2, 2, 64)
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    idx = [torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)]
    for call in (lambda: q4k.rope(x, idx[1], torch.zeros(4, 64)), lambda: q4k.kv_append(x, x, kc, kc, *idx),
                 lambda: q4k.paged_attention(x, kc, kc, *idx)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
