import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built q4k library")


@pytest.fixture(scope="session")
def oracle_mod():
    import oracle
    oracle.build()
    return oracle


@pytest.fixture(autouse=True)
def no_collection_in_captures(request, monkeypatch):
    """Destroying a CUDA graph invalidates every capture that is under way, and a graph that a test leaves in a cycle (a
    kept exception reaches its frames) is destroyed whenever the collector runs.  So it does not run inside
    torch.cuda.graph."""
    if request.node.get_closest_marker("gpu") is None:
        yield
        return
    import torch
    enter, leave = torch.cuda.graph.__enter__, torch.cuda.graph.__exit__

    def paused(self):
        gc.disable()
        try:
            return enter(self)
        except BaseException:
            gc.enable()
            raise

    def resumed(self, *exc):
        try:
            return leave(self, *exc)
        finally:
            gc.enable()

    monkeypatch.setattr(torch.cuda.graph, "__enter__", paused)
    monkeypatch.setattr(torch.cuda.graph, "__exit__", resumed)
    yield
