"""The C-ABI layer of the 8-bit linear layers, the norm with rotation, the
convolution and the next tokens (layer_api.hip) built as host C++ under AddressSanitizer
and UBSan, with stub launchers, driven with random valid and invalid calls on
the CPU.  Any sanitizer report fails the test."""
import os
import subprocess
import sys

import pytest

from tests.test_abi_sanitized import GXX, HERE, ROOT, sanitizer_runtime


@pytest.mark.skipif(GXX is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"),
                    reason="needs g++ and the HIP headers")
def test_entry_points_under_asan_and_ubsan(tmp_path):
    asan = sanitizer_runtime()
    if asan is None:
        pytest.skip("no libasan for g++")
    flags = ["-std=c++17", "-O1", "-g", "-fPIC", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include",
             "-I" + os.path.join(ROOT, "include")]
    csrc, here = os.path.join(ROOT, "bit_linear_layer_amd", "csrc"), os.path.join(HERE, "sanitize")
    objs = []
    for src in (os.path.join(csrc, "api.hip"), os.path.join(csrc, "layer_api.hip"),
                os.path.join(here, "stub_launchers.cpp"), os.path.join(here, "layer_stubs.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run([GXX, *flags, "-x", "c++", "-c", src, "-o", obj], check=True)
        objs.append(obj)
    lib = str(tmp_path / "libnvfp4_layers_sanitized.so")
    subprocess.run([GXX, "-shared", "-fsanitize=address,undefined", *objs, "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", lib], check=True)
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, os.path.join(here, "layer_driver.py"), lib], env=env, capture_output=True,
                       text=True, timeout=300)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-4000:]
    assert "sanitized layer driver ok" in r.stdout
    assert "ERROR: AddressSanitizer" not in report and "runtime error" not in report
