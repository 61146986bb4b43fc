"""The argument checks and plans of the 8-bit entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, as in test_sanitizers).  CPU only."""

import os
import subprocess

import pytest

from test_sanitizers import CLANG, PKG, ROOT, SAN, _run, build


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang++ not found")
def test_int8_validation_under_host_sanitizers(tmp_path):
    objdir = os.path.join(PKG, "_build")
    instrumented = ["mxq_api.hip", "gemm_int8.hip"]    # the checks, and the plans of the product
    others = [os.path.join(objdir, os.path.splitext(s)[0] + ".o") for s in build.SOURCES if s not in instrumented]
    if not all(os.path.exists(o) for o in others):
        build.build()
    flags = [f for f in build.FLAGS if f != "-shared"]
    host_san = [x for f in SAN for x in ("-Xarch_host", f)]
    objs = []
    for src in instrumented:
        objs.append(str(tmp_path / (src + ".o")))
        _run([build.hipcc(), *flags, "-O1", "-g", *host_san, "-c", "-o", objs[-1], os.path.join(build.CSRC, src)])
    drv = str(tmp_path / "int8_checks.o")
    _run([CLANG, "-std=c++17", "-O1", "-g", *SAN, "-c", "-o", drv, os.path.join(ROOT, "tests", "sanitize", "int8_checks.cpp")])
    exe = str(tmp_path / "int8_checks")
    rocm_lib = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "lib")
    _run([CLANG, *SAN, "-o", exe, drv, *objs, *others, "-L" + rocm_lib, "-lamdhip64", "-Wl,-rpath," + rocm_lib])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert " 0 failures" in out and "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
