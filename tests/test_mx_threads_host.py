"""First calls from several threads at once: what the launchers keep per device has no data race (thread sanitizer, on a
host stand-in for the CUDA runtime)."""
import os
import shutil
import subprocess

import pytest

from tests.fake_cuda import ROOT, cuda_include


def test_first_launches_from_several_threads(tmp_path):
    from gemm_uq_gb300.build import ARCH, CSRC, _nvcc
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    try:
        nvcc = _nvcc()
    except RuntimeError:
        pytest.skip("nvcc not found")
    hello = tmp_path / "hello.cpp"
    hello.write_text("int main() { return 0; }\n")
    exe = str(tmp_path / "hello")
    if subprocess.run([gxx, "-fsanitize=thread", "-o", exe, str(hello)], capture_output=True).returncode != 0 or \
            subprocess.run([exe], capture_output=True).returncode != 0:
        pytest.skip("no thread sanitizer here")
    jobs = []
    sources = [os.path.join(CSRC, "uq_mx_gemm.cu"), os.path.join(CSRC, "uq_moe.cu"), os.path.join(ROOT, "tests", "mx_threads_probe.cu")]
    for i, source in enumerate(sources):
        # the device code is not run: compiled without optimization, for speed
        jobs.append(subprocess.Popen([nvcc, *ARCH, "-Xptxas", "-O0", "-O1", "-g", "-std=c++17", "-Xcompiler",
                                      "-fPIC,-fsanitize=thread", "--expt-relaxed-constexpr", "-c", source, "-o",
                                      str(tmp_path / f"{i}.o")],
                                     stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for j in jobs:
        out, _ = j.communicate()
        assert j.returncode == 0, out[-3000:]
    exe = str(tmp_path / "probe")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-I", cuda_include(), "-o", exe,
                        os.path.join(ROOT, "tests", "fake_cudart.cpp"), *(str(tmp_path / f"{i}.o") for i in range(len(sources))),
                        "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "data race" not in r.stderr, r.stderr[:4000]
