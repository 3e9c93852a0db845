"""The attention tests once more for each form of the kernels, which small calls would not take by themselves: tiles of 8,
16 and 32 rows by clusters and split over the GPU, tiles of 256 rows on tcgen05.  A call that a form does not take (its
types, dim or pages) is refused and goes the library's way."""
import pytest

torch = pytest.importorskip("torch")
import test_attention_failure_gpu as failure   # noqa: E402
import test_attention_gpu as base              # noqa: E402
from test_attention_failure_gpu import test_dependent_launches_are_equal, test_wait_runs_out_then_recovers   # noqa: E402,F401
from test_attention_gpu import (test_bad_indices_are_not_followed, test_cap_and_bias, test_flat_and_peaked_scores,   # noqa: E402,F401
                                test_heads_and_dims, test_large_groups, test_lengths, test_long, test_masks,
                                test_offsets_past_32_bits, test_page_sizes, test_scales, test_scores_off_the_scale, test_types)

pytestmark = pytest.mark.gpu
FORMS = ["cluster8", "cluster16", "cluster32", "split8", "split16", "split32", "many"]


def _takes(form, q, kc, out_dtype, scale):
    dim, page = kc.shape[3], kc.shape[1]
    if form == "many":
        out = q.dtype if out_dtype is None else out_dtype
        return (q.dtype == kc.dtype and out != base.F32 and dim <= 128 and page % 16 == 0 and (scale is None or scale >= 0)
                and q.shape[1] // kc.shape[2] <= 256)
    return dim <= 128 or not form.endswith("32")


class _Formed:
    """The package with one form of attention."""

    def __init__(self, package, form):
        self._package, self._form, self.taken = package, form, 0

    def __getattr__(self, name):
        return getattr(self._package, name)

    def paged_attention(self, q, kc, vc, pt, start, ln, out=None, **kw):
        call = self._package.paged_attention
        dt = kw.get("out_dtype") or (None if out is None else out.dtype)
        if _takes(self._form, q, kc, dt, kw.get("scale")):
            self.taken += 1
            return call(q, kc, vc, pt, start, ln, out, form=self._form, **kw)
        if not kw.get("test_stall"):
            with pytest.raises(self._package.Q4KError) as e:
                call(q, kc, vc, pt, start, ln, out, form=self._form, **kw)
            assert e.value.status == 1
        return call(q, kc, vc, pt, start, ln, out, **kw)


@pytest.fixture(params=FORMS)
def q4k(request):
    import __graft_entry__
    __graft_entry__.build()
    import q4_dequant_gemv_gb300 as package
    torch.cuda.set_device(0)
    package.device_error_clear()
    return _Formed(package, request.param)


def test_form_names(q4k):
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    args = (q, kc, kc, base._dev([[0]]), base._dev([0, 1]), base._dev([1]))
    with pytest.raises(ValueError):
        q4k._package.paged_attention(*args, form="other")
    assert not q4k.paged_attention(*args).any() and q4k.taken == 1


@pytest.mark.parametrize("new,lens", [([1] * 40, [70 + 13 * i for i in range(40)]), ([8] * 24, [20 + 9 * i for i in range(24)]),
                                      ([600], [600]), ([7, 300, 0, 64], [1500, 300, 80, 900])])
@pytest.mark.parametrize("types", [(base.BF16,) * 3, (base.F32, base.F16, base.F32)])
def test_many_tiles(q4k, new, lens, types):
    """More tiles than fit at once."""
    base._run(q4k, dict(new=new, len=lens), 28, 4, 64, 16, *types)


@pytest.mark.parametrize("shape", [(torch.bfloat16, 2, 3, 700, 32), (torch.bfloat16, 1, 200, 700, 16)])
def test_stalls_of_16_bit_calls(q4k, shape):
    failure.test_wait_runs_out_then_recovers(q4k, shape)
