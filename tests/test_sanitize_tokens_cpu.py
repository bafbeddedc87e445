"""The token path's boundary (tokens_api.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_sanitize_cpu.py runs the scans': its host
code recompiled with the checks, linked with the other objects of the last
build, and its contract tests run in a child process, every report fatal.
"""
import os
import subprocess
import sys
import tempfile

import pytest

from scan_linear_rnns_amd import build as mgs_build
from tests.test_sanitize_cpu import CHECKS, CLANG, HOST_CHECKS, ROOT, _objects


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang not installed")
def test_tokens_abi_under_sanitizers():
    rt = subprocess.run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True,
                        check=True).stdout.strip()
    _objects()   # rebuilt if stale
    objs = [os.path.join(mgs_build.OBJ_DIR, o + ".o") for (_, o, _) in mgs_build.SOURCES if o != "tokens_api"]
    with tempfile.TemporaryDirectory(prefix="mgs_san_") as tmp:
        api = os.path.join(tmp, "tokens_api_san.o")
        cmd = mgs_build.compile_cmd(os.path.join(mgs_build.CSRC, "tokens_api.cpp"), api, ["-g", *HOST_CHECKS])
        subprocess.run(cmd, check=True, capture_output=True)
        lib = os.path.join(tmp, "libmgs_san.so")
        subprocess.run([CLANG + "++", "-shared", "-fPIC", *CHECKS, "-o", lib, api, *objs, "-L/opt/rocm/lib",
                        "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True, capture_output=True)
        env = dict(os.environ, LD_PRELOAD=rt, MGS_LIBRARY=lib, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
                   UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_tokens_abi_cpu.py"),
                            "-m", "not gpu", "-q", "-x", "-p", "no:cacheprovider"], env=env, cwd=ROOT,
                           capture_output=True, text=True, timeout=600)
        out = r.stdout + r.stderr
        assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
        assert r.returncode == 0 and " passed" in out, out[-4000:]
