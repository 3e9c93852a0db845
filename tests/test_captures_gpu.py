"""Graph captures: a graph left over from an earlier test does not disturb the next capture, and a
process may capture its first call."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_garbage_graphs_do_not_end_a_capture():
    """A captured graph in a cycle, then a capture whose body makes the collector run many times over."""
    x = torch.zeros(8, device="cuda")
    old = torch.cuda.CUDAGraph()
    with torch.cuda.graph(old):
        x.add_(1.0)
    cycle = {"graph": old}
    cycle["self"] = cycle
    del old, cycle
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1.0)
        kept = [[i] for i in range(200000)]
        x.add_(1.0)
    assert len(kept) == 200000
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, torch.full_like(x, 2.0))


FIRST = """
import sys
import torch
sys.path.insert(0, {root!r})
import q4_dequant_gemv_gb300 as q4k
g = torch.Generator(device="cuda").manual_seed(1)
q = torch.randn(40, 8, 64, generator=g, device="cuda").bfloat16()
kc, vc = (torch.randn(64, 16, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
pt = torch.randperm(64, generator=g, device="cuda").to(torch.int32).view(1, 64)
start, ln = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 40], [1000]))
table, pos = torch.rand(1024, 64, generator=g, device="cuda"), torch.arange(40, dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = q4k.paged_attention(q4k.rope(q, pos, table), kc, vc, pt, start, ln, form={form!r})
for _ in range(3):
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, q4k.paged_attention(q4k.rope(q, pos, table), kc, vc, pt, start, ln, form={form!r}))
assert q4k.device_error_flags() == 0
print("captured")
"""


@pytest.mark.parametrize("form", [None, "cluster16", "split8", "many"])
def test_first_call_of_a_process_is_captured(form):
    """What a first call sets up (attributes, the scratch pool, symbols) is set up inside the capture too."""
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, form=form)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr
