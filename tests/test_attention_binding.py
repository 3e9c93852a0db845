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
        self.shape, self.dtype = tuple(shape), dtype
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")
        self.is_cuda, self.recorded, self.allocated_on = device >= 0, [], stream
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
        return self.device.index if self.is_cuda else -1

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
        monkeypatch.setattr(_attention, "_device", lambda: self.device)
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


def _swaps(world):
    """(argument, call with that argument on another device) of every tensor argument."""
    x, k = (lambda d=0: Tensor((4, 2, 64), device=d)), (lambda d=0: Tensor((4, 2, 64), device=d))
    yield "pos", lambda: world.rope(pos=Tensor((4,), I32, 1))
    yield "table", lambda: world.rope(table=Tensor((8, 64), device=1))
    yield "y", lambda: world.rope(y=x(1))
    cache, index = world.cache(), world.index()
    base = [k(), k(), *cache, *index]
    names = ["k", "v", "k_cache", "v_cache", "page_table", "seq_start", "kv_len"]
    other = [k(1), k(1), *world.cache(1), *world.index(1)]
    for i in range(1, 7):
        yield "append " + names[i], lambda i=i: world.append(*base[:i], other[i], *base[i + 1:])
    yield "append pos", lambda: world.append(*base, table=Tensor((8, 64)), pos=Tensor((4,), I32, 1))
    yield "append table", lambda: world.append(*base, table=Tensor((8, 64), device=1))
    yield "append q", lambda: world.append(*base, q=x(1))
    yield "append q_out", lambda: world.append(*base, q=x(), q_out=x(1))
    base, other = [x(), *cache, *index], [x(1), *world.cache(1), *world.index(1)]
    names = ["q"] + names[2:]
    for i in range(1, 6):
        yield "attention " + names[i], lambda i=i: world.attention(*base[:i], other[i], *base[i + 1:])
    for name, t in (("out", x(1)), ("slopes", Tensor((2,), device=1)), ("prefix_len", Tensor((1,), I32, 1)),
                    ("kv_start", Tensor((4,), I32, 1)), ("lse", Tensor((4, 2), device=1))):
        yield "attention " + name, lambda name=name, t=t: world.attention(*base, **{name: t})


def test_tensors_of_several_devices_are_refused(world):
    """Before anything is launched: one device's kernel would follow another one's addresses."""
    for name, f in _swaps(world):
        with pytest.raises(ValueError, match="cuda:1"):
            f()
        assert not world.calls, name


def test_tensors_of_a_device_that_is_not_current_are_refused(world):
    """The library launches on the current device."""
    calls = [lambda: world.rope(Tensor((4, 2, 64), device=1), Tensor((4,), I32, 1), Tensor((8, 64), device=1)),
             lambda: world.append(Tensor((4, 2, 64), device=1), Tensor((4, 2, 64), device=1), *world.cache(1), *world.index(1)),
             lambda: world.attention(Tensor((4, 2, 64), device=1), *world.cache(1), *world.index(1))]
    for f in calls:
        with pytest.raises(ValueError, match="current device"):
            f()
        assert not world.calls
    world.device = 1
    for f in calls:
        f()
    assert [c[0] for c in world.calls] == ["rope", "append", "attention"]


def test_host_tensors_are_refused(world):
    for f in (lambda: world.rope(pos=torch.zeros(4, dtype=I32)), lambda: world.rope(x=Tensor((4, 2, 64), device=-1))):
        with pytest.raises((TypeError, ValueError)):
            f()
    assert not world.calls


def test_limits_past_32_bits_are_refused(world):
    """wait_limit_us is 32 bits wide in the library; 2^32 would be 0, which stands for two seconds."""
    for limit in (2 ** 32, 2 ** 40 + 5, -1):
        with pytest.raises((ValueError, OverflowError)):
            world.attention(wait_limit_us=limit)
    assert not world.calls
    world.attention(wait_limit_us=2 ** 32 - 1)
    assert [c[0] for c in world.calls] == ["attention"]
