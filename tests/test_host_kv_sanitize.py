"""The host code of the key-value cache's entry points under AddressSanitizer
and UndefinedBehaviorSanitizer, on the CPU: tests/sanitize/attention_check.cpp
makes their refusals, and checks the plan and the division by the page size."""
import glob
import os
import subprocess

from tensor_compiler_tiling_amd import build as B


def _stale() -> bool:
    if not os.path.exists(B.ATTENTION_CHECK):
        return True
    t = os.path.getmtime(B.ATTENTION_CHECK)
    srcs = glob.glob(os.path.join(B.CSRC, "*")) + [B.ATTENTION_CHECK_SRC, os.path.join(B.ROOT, "include", "convtile.h")]
    return any(os.path.getmtime(s) > t for s in srcs)


def test_attention_host_code_under_sanitizers():
    if _stale():
        B.build_host_check()
    env = dict(os.environ)
    # the HIP runtime's own allocations at process exit are not the library's
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    r = subprocess.run([B.ATTENTION_CHECK], capture_output=True, text=True, timeout=600, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "attention checks: 0 failed" in r.stdout
    assert "AddressSanitizer" not in out and "runtime error" not in out
