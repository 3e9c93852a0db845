"""q4k_scratch_keep without a GPU: its refusals, and its calls over a runtime that runs nothing."""
import ctypes

import pytest

from fake_runtime import fake, fake_path   # noqa: F401


def test_sizes_that_are_refused():
    from q4_dequant_gemv_gb300 import _build
    _build.build()
    import q4_dequant_gemv_gb300 as q4k
    assert q4k.raw_call("q4k_scratch_keep", -1) == 1
    for bad in (-1, 2 ** 63, 2 ** 64):
        with pytest.raises(ValueError):
            q4k.scratch_keep(bad)
    with pytest.raises(TypeError):
        q4k.scratch_keep("1")


@pytest.mark.parametrize("name", ["cudaMemPoolCreate", "cudaMemPoolSetAttribute"])
def test_a_failure_is_not_kept(fake, name):   # noqa: F811
    keep = fake.L.q4k_scratch_keep
    keep.argtypes = [ctypes.c_int64]
    for d in (0, 2, 0):
        fake.device(d)
        assert keep(1 << 30) == 0 and not fake.launches()
    fake.device(1)
    fake.fail(name)
    assert keep(0) == 4
    fake.fail(name, 0)
    assert keep(0) == 0 and keep(-1) == 1
