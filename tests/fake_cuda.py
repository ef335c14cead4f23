"""The library linked with a host stand-in for the CUDA runtime (fake_cudart.cpp): its launches are recorded, not run."""
import ctypes
import glob
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
Launch = namedtuple("Launch", "kernel grid block cluster overlap")


def cuda_include():
    from gemm_uq_gb300.build import _nvcc
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")


class FakeCuda:
    def __init__(self, path):
        import gemm_uq_gb300 as uq
        self.lib = ctypes.CDLL(path)
        for name, (res, args) in uq.SIGNATURES.items():
            fn = getattr(self.lib, name)
            fn.restype, fn.argtypes = res, args
        self.lib.fake_launch.restype = ctypes.c_char_p
        buf = (ctypes.c_uint8 * 4096)()
        self._keep = buf
        self.at = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256          # an aligned "device" address

    def launches(self, call):
        """The launches that call() makes; it has to return 0 (UQ_OK)."""
        self.lib.fake_clear()
        assert call() == 0, self.lib.uq_last_error()
        out = []
        for i in range(self.lib.fake_launch_count()):
            v = [ctypes.c_uint() for _ in range(3)] + [ctypes.c_int()]
            name = self.lib.fake_launch(i, *(ctypes.byref(x) for x in v)).decode()
            out.append(Launch(name, *(x.value for x in v)))
        return out


def load(tmp_path):
    """A library of its own per call: its state (workspaces, what is known of the device) starts empty."""
    from gemm_uq_gb300.build import BUILD, build
    build()
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    so = str(tmp_path / "libuq_fake.so")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", cuda_include(), "-o", so,
                        os.path.join(ROOT, "tests", "fake_cudart.cpp"), *sorted(glob.glob(os.path.join(BUILD, "*.o")))],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return FakeCuda(so)
