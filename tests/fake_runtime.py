"""The library's host code over a CUDA runtime that runs nothing (fake_cuda_runtime.cpp): what it launches, with which
sizes, on which device, and what it does when a call fails.  CPU only."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


class Launch(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char * 256), ("device", ctypes.c_int), ("grid", ctypes.c_int * 3), ("block", ctypes.c_int),
                ("smem", ctypes.c_int), ("cluster", ctypes.c_int), ("pdl", ctypes.c_int)]


class Library:
    """One loaded copy of the library, with state of its own."""

    def __init__(self, path):
        self.L = L = ctypes.CDLL(path, mode=ctypes.RTLD_LOCAL)
        P, S, I64 = ctypes.c_void_p, ctypes.c_char_p, ctypes.c_int64
        L.q4k_rope_table.argtypes = [P, I64, I64, S, P]
        L.q4k_rope.argtypes = [S, P]
        L.q4k_kv_append.argtypes = L.q4k_paged_attention.argtypes = [S, S, P]
        L.fake_launch.restype = ctypes.POINTER(Launch)
        L.fake_fail.argtypes = [S, ctypes.c_int, ctypes.c_int]

    def device(self, d):
        self.L.fake_set_device(d)

    def clusters(self, d, n):
        self.L.fake_set_clusters(d, n)

    def fail(self, name, times=1, skip=0):
        self.L.fake_fail(name.encode(), skip, times)

    def blocks(self, d):
        return self.L.fake_blocks(d)

    def launches(self):
        """The launches since the last call."""
        out = []
        for i in range(self.L.fake_launches()):
            out.append(Launch.from_buffer_copy(self.L.fake_launch(i).contents))
        self.L.fake_forget_launches()
        return out


@pytest.fixture(scope="session")
def fake_path(tmp_path_factory):
    from q4_dequant_gemv_gb300 import _build
    _build.build()
    objects = [os.path.join(_build.BUILD_DIR, os.path.basename(src)[:-3] + ".o") for src in _build._sources()]
    if not all(os.path.exists(o) for o in objects):
        _build.build(force=True)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    out = str(tmp_path_factory.mktemp("fake") / "libq4k_fake.so")
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", include, "-o", out,
                    os.path.join(HERE, "fake_cuda_runtime.cpp"), *objects, "-Wl,-Bsymbolic"], check=True)
    return out


@pytest.fixture
def fake(fake_path, tmp_path):
    """A fresh copy: nothing has been called in it."""
    path = str(tmp_path / "libq4k_fake.so")
    shutil.copy(fake_path, path)
    return Library(path)
