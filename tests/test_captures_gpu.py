"""Graph captures: a graph left over from an earlier test does not disturb the next capture."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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
