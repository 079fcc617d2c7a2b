"""The layer operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer: their
host-side suite in a child process against the host-sanitizer build of the library. No GPU is
used: the suite never launches a kernel."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc is needed to build the host-sanitizer library")
def test_layer_suite_under_address_and_undefined_behavior_sanitizers():
    from moe_grouped_gemm_fp32_amd import build

    lib = build.build_host_sanitized(verbose=False)
    env = dict(os.environ)
    env.update(LD_PRELOAD=build.sanitizer_runtime(), FP8GEMM_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                          "tests/test_layer_abi.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert " passed" in res.stdout
