"""The refusals of the serving operators' C-ABI layer, on the CPU: its host code
is compiled with AddressSanitizer and UndefinedBehaviorSanitizer against
stand-ins of the HIP runtime and of the launchers (host_serving_check.cpp), and
every refused call is seen to launch nothing."""

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_refusals_launch_nothing(tmp_path):
    from gguf_quant_block_amd import build
    exe = str(tmp_path / "check")
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-g", "-I", os.path.join(build.ROOT, "include"),
           "-I", build.CSRC, *build.SAN_HOST, os.path.join(HERE, "host_serving_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
