"""kda_layer_abi.cpp -- the argument checks, workspace layouts and the scan's plan of segments --
built with the host compiler against stand-in launchers (tests/sanitize/layer_stubs.cpp) under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only), and driven over many batches
(tests/sanitize/layer_driver.cpp).  Any report fails the test.
"""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-O1", "-g", "-fsanitize=address,undefined", "-fno-omit-frame-pointer", "-fno-sanitize-recover=all"]
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")


def _run(cmd, cwd):
    r = subprocess.run(cmd, cwd=cwd, capture_output=True, text=True, env=ENV)
    return r.returncode, r.stdout + r.stderr


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"), reason="needs g++ and HIP headers")
def test_layer_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "layer_asan")
    rc, out = _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(ROOT, "gated_delta_rule_log2_amd", "csrc", "kda_layer_abi.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "layer_stubs.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "layer_driver.cpp"),
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], str(tmp_path))
    assert rc == 0, out
    rc, out = _run([exe], str(tmp_path))
    assert rc == 0 and "layer driver ok" in out and "runtime error" not in out and "ERROR:" not in out, out
