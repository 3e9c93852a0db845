"""Appending to a cache whose slots or scales are one and the same (a stride of 0) is refused; reading and attention over such
scales are not.  Over a runtime that runs nothing."""
import pytest

pytest.importorskip("torch")
from fake_runtime import fake, fake_path   # noqa: F401,E402
from test_attention_abi import _attention   # noqa: E402
from test_cache8_abi import _append8, _bind, _cache8, _read8   # noqa: E402


@pytest.mark.parametrize("name", ["kp", "ks", "kh", "vp", "vs", "vh", "ksp", "ksb", "ksh", "vsp", "vsb", "vsh"])
def test_strides_of_zero(fake, name):   # noqa: F811
    L = _bind(fake)
    c = _cache8(**{name: 0})
    assert L.q4k_kv_append8(c, _append8(), 0) == 1 and not fake.launches()
    assert L.q4k_kv_read8(c, _read8(), 0) == 0
    assert L.q4k_paged_attention8(c, _attention(), 0) == 0


def test_strides_of_zero_that_no_index_uses(fake):   # noqa: F811
    L = _bind(fake)
    for c in (dict(pages=1, kp=0, vp=0, ksp=0, vsp=0), dict(heads=1, kh=0, vh=0, ksh=0, vsh=0), dict(size=4, ksb=0, vsb=0)):
        assert L.q4k_kv_append8(_cache8(**c), _append8(), 0) == 0, c
        assert fake.launches()
