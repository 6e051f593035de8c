"""The feed-forward calls' host code under AddressSanitizer and
UndefinedBehaviorSanitizer, without a GPU: tests/host/ffn_main.cpp drives it
against stand-ins for the kernel launchers that check every planned launch
(workspace regions inside the queried workspace and apart from one another,
tiles and units inside the matrix)."""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "bit_spherical_vector_amd", "csrc")
HOST = os.path.join(ROOT, "tests", "host")


def test_feed_forward_host_code_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("g++ or the ROCm headers are missing")
    exe = str(tmp_path / "svq_ffn_check")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-Wno-deprecated-declarations", "-o", exe]
    cmd += [os.path.join(CSRC, f) for f in ("svq_host.cpp", "svq_plan.cpp", "svq_ffn.cpp")]
    cmd += [os.path.join(HOST, f) for f in ("launch_checks.cpp", "ffn_checks.cpp", "ffn_main.cpp")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=900)
    assert res.returncode == 0, (res.stdout + res.stderr)[-4000:]
    assert "0 failures" in res.stdout
