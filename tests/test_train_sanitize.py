"""The host code behind include/muonstep_train.h under AddressSanitizer and UndefinedBehaviorSanitizer.

Like test_host_sanitize.py: the sanitizers are on the host code only, the driver is
tests/host_sanitize/exercise_train.c, and no GPU is used.
"""

import os
import subprocess

import pytest

from muon_optimizer_step_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang"


@pytest.mark.skipif(not (os.path.exists(build.HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not installed")
@pytest.mark.skipif(os.path.exists("/dev/kfd"),
                    reason="the test program's valid calls carry fake device pointers: run only where no GPU is present")
def test_host_code_is_clean_under_asan_and_ubsan(tmp_path):
    lib = tmp_path / "libmuonstep_san.so"
    flags = [f if f != "-O3" else "-O1" for f in build.FLAGS]
    cmd = [build.HIPCC, *flags, "-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-fno-sanitize-recover=undefined",
           *[os.path.join(build.CSRC, s) for s in build.SOURCES], "-o", str(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    exe = tmp_path / "exercise_train"
    r = subprocess.run([CLANG, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                        "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "host_sanitize", "exercise_train.c"),
                        f"-L{tmp_path}", "-lmuonstep_san", f"-Wl,-rpath,{tmp_path}", "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    # the HIP runtime the library loads is not instrumented and keeps allocations for the process lifetime
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "ALL OK" in r.stdout, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
