"""The Python calls of the attention operators over stand-ins for tensors, streams and the library: which memory an
output gets, which devices a call takes.  CPU only; nothing is launched."""
import contextlib
import ctypes
import types

import pytest

torch = pytest.importorskip("torch")
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


class Stream:
    def __init__(self, name, handle, device=0):
        self.name, self.cuda_stream, self.device = name, handle, device


class Tensor:
    """What the calls read of a CUDA tensor."""

    def __init__(self, shape, dtype=F32, device=0, stream=None, strides=None):
        self.shape, self.dtype, self.device = tuple(shape), dtype, torch.device("cuda", device)
        self.is_cuda, self.recorded, self.allocated_on = True, [], stream
        self._strides = strides

    def stride(self):
        if self._strides:
            return self._strides
        out, n = [], 1
        for s in reversed(self.shape):
            out.append(n)
            n *= s
        return tuple(reversed(out))

    def data_ptr(self):
        return 0x10000

    def is_contiguous(self):
        return self._strides is None

    def get_device(self):
        return self.device.index

    def record_stream(self, stream):
        self.recorded.append(stream)


class World:
    """A package whose torch and library are stand-ins: `now` is the current stream, `device` the current device."""

    def __init__(self, monkeypatch):
        import q4_dequant_gemv_gb300 as package
        from q4_dequant_gemv_gb300 import _attention, _build
        _build.build()
        self.calls, self.device = [], 0
        self.main, self.side = Stream("main", 0), Stream("side", 77)
        self.now = self.main

        def empty(shape, dtype=F32, device=None):
            return Tensor(shape, dtype, torch.device(device).index, self.now)

        def empty_like(x):
            return Tensor(x.shape, x.dtype, x.device.index, self.now)

        @contextlib.contextmanager
        def on(stream):
            before, self.now = self.now, stream
            try:
                yield
            finally:
                self.now = before

        @contextlib.contextmanager
        def device(d):
            before, self.device = self.device, torch.device(d).index
            try:
                yield
            finally:
                self.device = before

        cuda = types.SimpleNamespace(stream=on, device=device, current_stream=lambda d=None: self.now,
                                     current_device=lambda: self.device)
        monkeypatch.setattr(_attention, "torch", types.SimpleNamespace(
            Tensor=Tensor, float32=F32, float16=torch.float16, bfloat16=BF16, int32=I32, empty=empty, empty_like=empty_like,
            cuda=cuda, device=torch.device))
        monkeypatch.setattr(_attention, "_current", lambda d: self.now.cuda_stream)
        monkeypatch.setattr(_attention, "_device", lambda: self.device, raising=False)
        _attention._calls = None
        proto = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)
        proto3 = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)

        def note(name):
            return lambda *a: self.calls.append((name, a[-1] or 0)) or 0

        self.lib = types.SimpleNamespace(
            q4k_rope=proto(note("rope")), q4k_kv_append=proto3(note("append")), q4k_paged_attention=proto3(note("attention")),
            q4k_rope_table=lambda p, rows, rot, s, on: self.calls.append(("table", on)) or 0)
        monkeypatch.setattr(package, "lib", lambda: self.lib)
        self.m = _attention

    def rope(self, x=None, pos=None, table=None, **kw):
        x = Tensor((4, 2, 64)) if x is None else x
        return self.m.rope(x, Tensor((4,), I32) if pos is None else pos, Tensor((8, 64)) if table is None else table, **kw)

    def index(self, device=0):
        return [Tensor((1, 2), I32, device), Tensor((2,), I32, device), Tensor((1,), I32, device)]

    def cache(self, device=0):
        return [Tensor((3, 16, 2, 64), BF16, device) for _ in range(2)]

    def append(self, *a, **kw):
        a = a or (Tensor((4, 2, 64)), Tensor((4, 2, 64)), *self.cache(), *self.index())
        return self.m.kv_append(*a, **kw)

    def attention(self, *a, **kw):
        a = a or (Tensor((4, 2, 64)), *self.cache(), *self.index())
        return self.m.paged_attention(*a, **kw)


@pytest.fixture
def world(monkeypatch):
    yield World(monkeypatch)
    # the next call outside sets the compiled calls up again with torch itself
    import q4_dequant_gemv_gb300._attention as m
    m._calls = None


def _new_outputs(world, **kw):
    return {
        "rope": lambda: world.rope(**kw), "rope of another type": lambda: world.rope(out_dtype=BF16, **kw),
        "rope of a strided x": lambda: world.rope(x=Tensor((4, 2, 64), strides=(256, 128, 1)), **kw),
        "append": lambda: world.append(q=Tensor((4, 4, 64)), **kw), "attention": lambda: world.attention(**kw),
        "table": lambda: world.m.rope_table(16, 64, device=torch.device("cuda", 0), **kw),
    }


def test_outputs_are_the_calls_streams_own(world):
    """A block that the current stream has freed may still be read there, and only that stream's order makes it safe to
    take: an output that another stream writes comes from that stream's blocks.  The current stream, where the caller
    goes on with it, is told to the allocator."""
    for name, f in _new_outputs(world, stream=world.side).items():
        world.calls.clear()
        y = f()
        assert y.allocated_on is world.side, name
        assert world.main in y.recorded, name
        assert [c[1] for c in world.calls] == [77] and world.now is world.main, name


def test_outputs_of_the_current_stream(world):
    for now in (world.main, world.side):
        world.now = now
        for name, f in _new_outputs(world).items():
            world.calls.clear()
            y = f()
            assert y.allocated_on is now and not y.recorded, name
            assert [c[1] for c in world.calls] == [now.cuda_stream], name
