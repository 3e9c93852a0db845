"""Waits that run out in every form of the kernels, over several tiles and both kinds of masks: the kernel ends by itself,
says so, and what runs next on the same SMs is not disturbed by what was in flight."""
import time

import pytest

torch = pytest.importorskip("torch")
from test_attention_failure_gpu import _call   # noqa: E402
from test_attention_forms_gpu import FORMS, _takes   # noqa: E402
from test_attention_gpu import q4k   # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", [(torch.bfloat16, 2, 300, 2000, 64), (torch.bfloat16, 3, 2, 3000, 16), (torch.float32, 2, 20, 900, 32)])
@pytest.mark.parametrize("docs", [False, True])
def test_wind_down_leaves_nothing_in_flight(q4k, form, shape, docs):   # noqa: F811
    q, kc, *index = _call(*shape)
    if not _takes(form, q, kc, None, None):
        pytest.skip("the form does not take the call")
    kw = dict(form=form)
    if docs:        # a document that begins inside a unit of keys
        kw["kv_start"] = torch.full((q.shape[0],), 70, dtype=torch.int32, device="cuda")
    want = q4k.paged_attention(q, kc, *index, **kw)
    torch.cuda.synchronize()
    for limit in (1, 1000):
        t0 = time.time()
        for _ in range(3):      # (the launches after the first meet whatever it left behind)
            q4k.paged_attention(q, kc, *index, wait_limit_us=limit, test_stall=True, **kw)
        after = q4k.paged_attention(q, kc, *index, **kw)
        torch.cuda.synchronize()
        assert time.time() - t0 < 10.0
        assert q4k.device_error_flags() == 8
        q4k.device_error_clear()
        assert torch.equal(after, want)
    assert torch.equal(q4k.paged_attention(q, kc, *index, **kw), want)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
