"""What the workgroup-placement probe accepts, under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU (tests/sanitize/placement_check.cpp)."""
import glob
import os
import subprocess

from tensor_compiler_tiling_amd import build as B


def _stale() -> bool:
    if not os.path.exists(B.PLACEMENT_CHECK):
        return True
    t = os.path.getmtime(B.PLACEMENT_CHECK)
    srcs = glob.glob(os.path.join(B.CSRC, "*")) + [B.PLACEMENT_CHECK_SRC]
    return any(os.path.getmtime(s) > t for s in srcs)


def test_placement_under_sanitizers():
    if _stale():
        B.build_host_check()
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([B.PLACEMENT_CHECK], capture_output=True, text=True, timeout=600, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "placement checks: 0 failed" in r.stdout
    assert "AddressSanitizer" not in out and "runtime error" not in out
