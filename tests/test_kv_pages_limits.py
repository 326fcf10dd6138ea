"""The largest calls of the paged KV cache's entry points, on the CPU: the C-ABI
layer built as plain host C++ with stub launchers, so that a call that is
accepted launches nothing."""
import ctypes
import os
import subprocess

import pytest

import bit_linear_layer_amd as nv
from tests.test_abi_sanitized import GXX, HERE, ROOT
from tests.test_kv_pages_refusals import FAKE, pages

pytestmark = pytest.mark.skipif(GXX is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"),
                                reason="needs g++ and the HIP headers")
ROWS_OF_A_WORKGROUP, THREADS = 16, 256
GRID = 1 << 32  # a launch has fewer threads than this in each dimension


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("kv_limits")
    flags = ["-std=c++17", "-O1", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include")]
    objs = []
    for src in (os.path.join(ROOT, "bit_linear_layer_amd", "csrc", "api.hip"),
                os.path.join(ROOT, "bit_linear_layer_amd", "csrc", "kv_pages_api.hip"),
                os.path.join(HERE, "sanitize", "stub_launchers.cpp"), os.path.join(HERE, "sanitize", "kv_pages_stubs.cpp")):
        obj = str(tmp / (os.path.basename(src) + ".o"))
        subprocess.run([GXX, *flags, "-x", "c++", "-c", src, "-o", obj], check=True)
        objs.append(obj)
    out = str(tmp / "libkv_limits.so")
    subprocess.run([GXX, "-shared", *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", out], check=True)
    so = ctypes.CDLL(out)
    for name in ("nvfp4_kv_pages_write", "nvfp4_kv_pages_read"):
        getattr(so, name).argtypes = getattr(nv.load(), name).argtypes
    return so


@pytest.mark.parametrize("rows", [1, 16, (1 << 28) - 17, (1 << 28) - 16, (1 << 28) - 15, (1 << 28) - 1, 1 << 28])
def test_rows_fit_a_launch(lib, rows):
    p = pages()
    fits = -(-rows // ROWS_OF_A_WORKGROUP) * THREADS < GRID
    for call in (lambda: lib.nvfp4_kv_pages_write(ctypes.byref(p), FAKE, 256, FAKE, 256, 0, rows, FAKE, None),
                 lambda: lib.nvfp4_kv_pages_read(ctypes.byref(p), rows, FAKE, FAKE, 256, FAKE, 256, 0, None)):
        before = lib.nvfp4_kv_stub_calls()
        status = call()
        assert status == (0 if fits else -11)
        assert lib.nvfp4_kv_stub_calls() == before + fits
