"""The choice of the next token on the CPU: the C-ABI layer's refusals and workspace (host_sample_check.cpp, compiled with
AddressSanitizer and UndefinedBehaviorSanitizer against stand-ins), what the binding refuses, and the oracle's pins."""

import math
import os
import subprocess

import numpy as np
import pytest
import torch

from gguf_quant_block_amd import serving
from oracle import sampling as o

HERE = os.path.dirname(os.path.abspath(__file__))


def test_refusals_launch_nothing(tmp_path):
    from gguf_quant_block_amd import build
    exe = str(tmp_path / "check")
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-g", "-I", os.path.join(build.ROOT, "include"),
           "-I", build.CSRC, *build.SAN_HOST, os.path.join(HERE, "host_sample_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def test_binding(monkeypatch):
    calls = []
    monkeypatch.setitem(serving._calls, "fc_gguf_sample", lambda *a: calls.append(a) or 0)
    monkeypatch.setitem(serving._calls, "fc_gguf_sample_workspace", lambda rows, vocab: 16)
    monkeypatch.setattr(serving, "_workspaces", {})
    monkeypatch.setattr(serving, "_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    flat = torch.zeros(4096)
    x, u = flat[:200].view(2, 100), flat[200:202]
    serving.sample(x, u)
    assert calls[-1][:5] == (x.data_ptr(), 100, 2, 2, 100) and calls[-1][5] == u.data_ptr() and calls[-1][6:10] == (None,) * 4
    out, lp = flat[300:302].view(torch.int32), flat[302:304]
    assert serving.sample(x[:, :90], u, temperature=flat[310:312], min_p=flat[312:314], out=out, logprobs=lp) is out
    assert calls[-1][1] == 100 and calls[-1][4] == 90 and calls[-1][6] == flat[310:].data_ptr() and calls[-1][11] == lp.data_ptr()
    n = len(calls)
    for at in (0, 99, 198, 199, 200, 201):                     # among the logits and the random numbers
        with pytest.raises(ValueError):
            serving.sample(x, u, out=flat[at:at + 2].view(torch.int32))
        with pytest.raises(ValueError):
            serving.sample(x, u, logprobs=flat[at:at + 2])
    for kw in ({"temperature": lp}, {"top_k": lp.view(torch.int32)}, {"top_p": lp}, {"min_p": flat[303:305]}):
        with pytest.raises(ValueError):
            serving.sample(x, u, logprobs=lp, **kw)
    for bad in (flat[301:303], flat[300:302]):
        with pytest.raises(ValueError):
            serving.sample(x, u, out=out, logprobs=bad)
    with pytest.raises(ValueError):
        serving.sample(x.t(), u[:1].expand(100))
    assert len(calls) == n
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        serving.sample(x, u)
    assert len(calls) == n


def test_oracle():
    x = np.log([0.1, 0.4, 0.2, 0.2, 0.1])
    # order: 1, 2, 3, 0, 4
    for u, want in ((0.0, 1), (0.39, 1), (0.41, 2), (0.59, 2), (0.61, 3), (0.81, 0), (0.95, 4), (1.0, 4)):
        assert o.choose(x, u)[0] == want
    assert o.choose(x, 0.99, top_k=2)[0] == 2 and abs(o.choose(x, 0.99, top_k=2)[1] - math.log(1 / 3)) < 1e-12
    assert o.choose(x, 0.99, top_p=0.7)[2] == 3 and o.choose(x, 0.99, top_p=0.3)[2] == 1
    assert o.choose(x, 0.99, min_p=0.3)[2] == 3 and o.choose(x, 0.99, min_p=0.9)[2] == 1
    assert o.choose(x, 0.99, top_k=3, top_p=0.7)[2] == 2                # 0.7 of the 0.8 that three tokens hold
    assert o.choose(x, 0.99, temperature=0)[:2] == (1, 0.0)
    assert abs(o.choose(x, 0.0, temperature=0.5)[1] - math.log(0.16 / (0.16 + 0.08 + 0.02))) < 1e-12
    assert o.choose([-np.inf, np.nan], 0.5)[0] == -1 and o.choose([1.0, np.inf, np.inf], 0.75)[0] == 2
