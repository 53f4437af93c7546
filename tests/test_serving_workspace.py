"""The attention workspace against captured graphs (host_workspace_check.cpp) and the sizes that an attention call takes
(host_limits_check.cpp), on the CPU: the C-ABI layer and the library's own plan, compiled with AddressSanitizer and
UndefinedBehaviorSanitizer against stand-ins of the HIP runtime and of the launchers, which keep account of the memory
and of the grids."""

import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("check", ["host_workspace_check.cpp", "host_limits_check.cpp"])
def test_on_the_host(tmp_path, check):
    from gguf_quant_block_amd import build
    exe = str(tmp_path / "check")
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-g", "-I", os.path.join(build.ROOT, "include"),
           "-I", build.CSRC, *build.SAN_HOST, os.path.join(HERE, check), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
