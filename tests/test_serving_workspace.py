"""The attention workspace against captured graphs, on the CPU: the C-ABI layer and the library's own plan, compiled
with AddressSanitizer and UndefinedBehaviorSanitizer against stand-ins of the HIP runtime and of the launchers
(host_workspace_check.cpp), which keep account of the memory that launches use."""

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_launches_find_their_workspace(tmp_path):
    from gguf_quant_block_amd import build
    exe = str(tmp_path / "check")
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-g", "-I", os.path.join(build.ROOT, "include"),
           "-I", build.CSRC, *build.SAN_HOST, os.path.join(HERE, "host_workspace_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
