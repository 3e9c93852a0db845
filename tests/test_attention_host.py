"""Host side of the rotary, append and attention calls over a runtime that runs nothing: several devices, calls that fail,
strides that do not matter."""
import pytest

from fake_runtime import fake, fake_path   # noqa: F401
from test_attention_abi import OK, _append, _attention, _cache, _rope

FORMS = {"cluster8": 1, "cluster16": 2, "cluster32": 3, "split8": 4, "split16": 5, "split32": 6, "many": 7}


def _call(lib, form=0, cache=None, **kw):
    return lib.L.q4k_paged_attention(_cache(**(cache or {})), _attention(flags=form << 8, **kw), 0)


@pytest.mark.parametrize("form", FORMS)
def test_every_device_gets_what_it_needs(fake, form):   # noqa: F811
    """A kernel's shared memory limit, the scratch pool and the error word belong to a device."""
    for d in (0, 1, 0, 3, 1):
        fake.device(d)
        assert _call(fake, FORMS[form]) == 0, f"device {d}"
        assert all(x.device == d for x in fake.launches())
        assert fake.blocks(d) == 0


def test_clusters_that_fit_are_a_devices_own(fake):   # noqa: F811
    """A device that holds no cluster takes the split, one that does goes on taking clusters."""
    fake.clusters(1, 0)
    for d in (0, 1, 0):
        fake.device(d)
        assert _call(fake) == 0
        kernels = fake.launches()
        if d == 1:
            assert len(kernels) == 2 and kernels[0].cluster == 0 and b"join" in kernels[1].kernel
        else:
            assert len(kernels) == 1 and kernels[0].cluster >= 1


@pytest.mark.parametrize("form", ["cluster8", "split8", "many"])
@pytest.mark.parametrize("name", ["cudaFuncSetAttribute", "cudaOccupancyMaxActiveClusters", "cudaMemPoolCreate",
                                  "cudaMemPoolSetAttribute", "cudaMallocFromPoolAsync", "cudaGetSymbolAddress",
                                  "cudaLaunchKernelExC"])
def test_a_failure_is_not_kept(fake, form, name):   # noqa: F811
    """The call that meets it says so and leaves nothing behind; the next one works."""
    fake.fail(name)
    pool = "MemPool" in name or "FromPool" in name
    assert _call(fake, FORMS[form]) == (0 if pool and form == "cluster8" else 4)
    assert fake.blocks(0) == 0
    fake.fail(name, 0)
    fake.launches()
    assert _call(fake, FORMS[form]) == 0
    assert fake.launches() and fake.blocks(0) == 0


@pytest.mark.parametrize("form", ["split8", "many"])
def test_a_join_that_fails_gives_its_scratch_back(fake, form):   # noqa: F811
    fake.fail("cudaLaunchKernelExC", skip=1)
    assert _call(fake, FORMS[form]) == 4
    assert len(fake.launches()) == 1 and fake.blocks(0) == 0


@pytest.mark.parametrize("cache,call", [
    (dict(pages=1, kp=2051), {}), (dict(size=1, ks=67, vs=3), {}), (dict(heads=1, kh=5, vh=7), dict(heads=1, qt=64, ot=64, qh=3, oh=9)),
    (dict(tokens=1), dict(qt=777, ot=1)), (dict(tokens=1, heads=1, pages=1, kp=-3, vp=1, kh=1, vh=3), dict(heads=1, qt=-5, ot=3, qh=1, oh=-1)),
])
def test_strides_that_no_index_uses(fake, cache, call):   # noqa: F811
    """Of an axis of one element: whatever they are, they make neither a refusal nor a difference to the launch."""
    plain = {k: v for k, v in cache.items() if k in ("pages", "size", "heads", "tokens")}
    assert _call(fake, cache=plain, **{k: v for k, v in call.items() if k == "heads"}) == 0
    want = [(x.kernel, x.grid[:], x.smem) for x in fake.launches()]
    assert _call(fake, cache=cache, **call) == 0
    assert [(x.kernel, x.grid[:], x.smem) for x in fake.launches()] == want


def test_strides_that_no_index_uses_in_rope_and_append(fake):   # noqa: F811
    """They do not send a call to the element-wise kernel."""
    for kw in (dict(tokens=1, xt=1, yt=-7), dict(heads=1, xh=3, yh=5, xt=64, yt=64)):
        assert fake.L.q4k_rope(_rope(**kw), 0) == 0
        assert [b"wide_kernel" in x.kernel for x in fake.launches()] == [True]
    for cache, kw in ((dict(pages=1, kp=2051, vp=1), {}), (dict(size=1, ks=67, vs=3), {}), (dict(heads=1, kh=5, vh=7), dict(kh=3, vh=1)),
                      (dict(tokens=1), dict(kt=5, vt=7)), (dict(tokens=1), dict(q=OK, qo=OK, heads=1, qt=3, qh=1, ot=1, oh=5))):
        assert fake.L.q4k_kv_append(_cache(**cache), _append(**kw), 0) == 0
        assert [b"wide_kernel" in x.kernel for x in fake.launches()] == [True], (cache, kw)
    # .. where an index uses them they do
    assert fake.L.q4k_rope(_rope(xt=193), 0) == 0
    assert [b"narrow_kernel" in x.kernel for x in fake.launches()] == [True]
