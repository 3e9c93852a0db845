"""Calls on another stream than the current one."""
import pytest

torch = pytest.importorskip("torch")
from test_attention_failure_gpu import _call, q4k   # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_outputs_take_no_memory_that_is_in_use(q4k):   # noqa: F811
    """Memory freed on the current stream, which has still to read it, is not what a call on a side stream writes."""
    q, kc, vc, pt, start, ln = _call(torch.float32, 2, 40, 60, 16)
    k, v = q[:, :2].contiguous(), q[:, 2:4].contiguous()
    table, pos = q4k.rope_table(128, 64), torch.arange(80, dtype=torch.int32, device="cuda")
    calls = [lambda **kw: q4k.rope(q, pos, table, **kw),
             lambda **kw: q4k.kv_append(k, v, kc, vc, pt, start, ln, table=table, q=q, **kw),
             lambda **kw: q4k.paged_attention(q, kc, vc, pt, start, ln, **kw),
             lambda **kw: q4k.rope_table(80 * 8, 64, device=q.device, **kw).view(80, 8, 64)]
    side = torch.cuda.Stream()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        for _ in range(2):      # (the second time round the side stream has freed blocks of its own)
            old = torch.full_like(want, 5.0)
            at = old.data_ptr()
            torch.cuda._sleep(100000000)
            late = old.clone()
            del old
            y = call(stream=side)
            assert y.data_ptr() != at
            side.synchronize()
            assert torch.equal(y, want)
            torch.cuda.synchronize()
            assert torch.all(late == 5.0)
            del y
    assert q4k.device_error_flags() == 0
