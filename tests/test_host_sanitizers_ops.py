"""The argument checks of the 4-bit operators and the mixture-of-experts layer (ops.cpp) under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only).

ops.cpp is compiled by the host compiler with the rest of the library's host
code and every report fatal; the launchers are stand-ins (tests/host_sanitize).
The refusal tests and calls at the limits of the arguments run against that
library in a child process.  No GPU code is built or run.
"""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_tile_signaling_amd", "csrc")

LIMITS = """
import ctypes as C, itertools
import gemm_tile_signaling_amd as fo
from gemm_tile_signaling_amd import moe
o = moe._ops()
edges = [-2 ** 63, -1, 0, 1, 8, 32, 2 ** 20, 2 ** 31 - 8, 2 ** 31, 2 ** 40, 2 ** 63 - 32, 2 ** 63 - 1]
p = 4096                    # an aligned address that nothing reads
calls = 0
for a, b, c in itertools.product(edges, repeat=3):
    for t in (-1, 0, 1, 2, 3):
        rc = {o.fo_mx4_quantize(p, a, b, c, t, p, p, None), o.fo_mx4_dequantize(p, p, a, b, t, p, None),
              o.fo_mx4_gemm(p, p, p, p, p, a, b, c, t, 1, None, None)}
        assert rc <= {fo.FO_OK, fo.FO_ERR_INVALID, fo.FO_ERR_UNSUPPORTED, fo.FO_ERR_HIP}, rc
        calls += 3
small = [-2 ** 31, -1, 0, 1, 16, 64, 1024, 2 ** 31 - 1]
n = C.c_int64()
for a, b in itertools.product(edges, repeat=2):
    for e, k, first, local in itertools.product(small, small[2:5], small, small):
        d = moe._MoeDesc(a, b, e, k, first, local, 0, 1, 1, 64)
        if o.fo_moe_workspace_bytes(C.byref(d), C.byref(n)) == fo.FO_OK:
            assert 0 < n.value < 2 ** 40
        calls += 1
print("calls", calls)
"""


def _build(out):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not available")
    asan = subprocess.run([gxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not asan or not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("the AddressSanitizer runtime is not available")
    srcs = [os.path.join(CSRC, f) for f in ("plan.cpp", "search.cpp", "api.cpp", "ops.cpp")]
    srcs += [os.path.join(ROOT, "tests", "host_sanitize", f) for f in ("launch_stubs.cpp", "ops_stubs.cpp")]
    cmd = [gxx, "-std=c++17", "-shared", "-fPIC", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), *srcs, "-o", out,
           "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return asan


@pytest.mark.slow
def test_refusals_and_limits_under_sanitizers(tmp_path):
    lib = str(tmp_path / "libfo_ops_sanitized.so")
    asan = _build(lib)
    env = dict(os.environ, FO_LIB=lib, LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    for args in (["-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider", "tests/test_mx4_refusals.py",
                  "tests/test_moe_refusals.py"], ["-c", LIMITS]):
        r = subprocess.run([sys.executable, *args], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
        out = r.stdout[-3000:] + r.stderr[-3000:]
        assert r.returncode == 0, out
        assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out
        assert " passed" in r.stdout or "calls" in r.stdout, out
