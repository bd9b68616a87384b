"""The host rules of the gated block and of 4-bit weights (csrc/gated_host.cpp, csrc/w4_host.cpp and
csrc/plan_host.cpp below them) built with g++ under AddressSanitizer and UndefinedBehaviorSanitizer
and run through tests/sanitize/gated_driver.cpp. Any sanitizer report or failed check fails the
test."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "gemm_epilogues_epilog_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_host_rules_under_asan_and_ubsan(tmp_path):
    exe = tmp_path / "gated_sanitized"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-Wall", "-Wextra",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           *(os.path.join(CSRC, f) for f in ("gated_host.cpp", "w4_host.cpp", "plan_host.cpp")),
           os.path.join(HERE, "sanitize", "gated_driver.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "ok (0 failures)" in r.stdout, r.stdout[-3000:] + r.stderr[-4000:]
