"""Failure path of the attention kernels' bounded waits, made to run out without any fault: the test-only stall flag
has the first copy of each CTA awaited for 16 bytes more than it brings, with a bound of 1 ms.  The kernel returns by
itself, sets its bit, leaves the context usable, and the next call gives what an undisturbed one gave.  And: calls
launched as programmatic dependents give the same bits as plain ones."""
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4k():
    import __graft_entry__
    __graft_entry__.build()
    import q4_dequant_gemv_gb300 as q4k
    torch.cuda.set_device(0)
    q4k.device_error_clear()
    return q4k


def _call(dtype, batch, n, past, page, heads=8, kv_heads=2, dim=64, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = past + n
    per = -(-total // page)
    q = torch.randn(batch * n, heads, dim, generator=g, device="cuda").to(dtype)
    kc, vc = (torch.randn(batch * per, page, kv_heads, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pt = torch.randperm(batch * per, generator=g, device="cuda").to(torch.int32).view(batch, per)
    start = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n
    return q, kc, vc, pt, start, torch.full((batch,), total, dtype=torch.int32, device="cuda")


# clusters that share a tile (one row tile, two), the split over all CTAs, the tcgen05 kernel
CALLS = [(torch.float32, 1, 1, 500, 16), (torch.float32, 3, 5, 200, 16), (torch.float32, 1, 1, 100000, 64),
         (torch.bfloat16, 2, 200, 700, 32)]


@pytest.mark.parametrize("shape", CALLS)
def test_wait_runs_out_then_recovers(q4k, shape):
    args = _call(*shape)
    want = q4k.paged_attention(*args)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0
    t0 = time.time()
    q4k.paged_attention(*args, wait_limit_us=1000, test_stall=True)
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert q4k.device_error_flags() == 8
    q4k.device_error_clear()
    assert q4k.device_error_flags() == 0
    assert torch.equal(q4k.paged_attention(*args), want)
    torch.cuda.synchronize()
    assert q4k.device_error_flags() == 0


@pytest.mark.parametrize("shape", CALLS + [(torch.float32, 2, 3, 40, 5)])
def test_dependent_launches_are_equal(q4k, shape):
    """rope, append and attention in a row on one stream and in a graph, each reading what the one before wrote."""
    q, kc, vc, pt, start, ln = _call(*shape)
    n = q.shape[0]
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(n, 2, 64, generator=g, device="cuda") for _ in range(2))
    table = q4k.rope_table(int(ln.max()), 64)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    kw = dict(wait_limit_us=0)

    def chain(pdl):
        a = q4k.rope(q, pos, table, pdl=pdl)
        b = q4k.kv_append(k, v, kc, vc, pt, start, ln, table=table, q=a, pdl=pdl)
        c = q4k.paged_attention(b, kc, vc, pt, start, ln, pdl=pdl, **kw)
        return q4k.rope(c, pos, table, pdl=pdl)

    want = chain(False)
    for _ in range(3):
        assert torch.equal(chain(True), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(True)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert q4k.device_error_flags() == 0
