"""Norms and the cache of 8 bits on the CPU: the C-ABI layer's refusals (host_kv8_check.cpp, compiled with
AddressSanitizer and UndefinedBehaviorSanitizer against stand-ins), what the binding hands to the library, and the
oracle's own pins."""

import os
import subprocess

import numpy as np
import pytest
import torch

from gguf_quant_block_amd import serving
from oracle import serving8 as o8

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("check", ["host_kv8_check.cpp"])
def test_refusals_launch_nothing(tmp_path, check):
    from gguf_quant_block_amd import build
    exe = str(tmp_path / "check")
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-g", "-I", os.path.join(build.ROOT, "include"),
           "-I", build.CSRC, *build.SAN_HOST, os.path.join(HERE, check), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def test_binding_hands_norms_over(monkeypatch):
    calls = []
    for name in ("fc_gguf_kv_append", "fc_gguf_kv_append_norm"):
        monkeypatch.setitem(serving._calls, name, lambda *a, name=name: calls.append((name, a)) or 0)
    monkeypatch.setattr(serving, "_stream", lambda index: 0)
    kv = object.__new__(serving.PagedKv)
    kv.index, kv.head_dim, kv.kv_heads, kv.page_size, kv.pages = -1, 64, 2, 16, 4
    kv.dtype, kv.device, kv.scale, kv._h = torch.float16, torch.device("cpu"), 0.125, None

    def norm(q, k):
        n = object.__new__(serving.HeadNorm)
        n.index, n.q, n.k, n.eps = -1, q, k, 1e-5
        n.q_shape, n.k_shape = (None if w is None else tuple(w.shape) for w in (q, k))
        n.q_ptr, n.k_ptr = (None if w is None else w.data_ptr() for w in (q, k))
        return n

    q, k = torch.zeros((3, 4, 64), dtype=torch.float16), torch.zeros((3, 2, 64), dtype=torch.float16)
    slots = torch.tensor([0, 1, 2], dtype=torch.int32)
    one, each = torch.ones(64), torch.ones((2, 64))
    at = slice(10, 15)                                       # q_norm, its stride, k_norm, its stride, eps
    for n, want in ((norm(one, each), (one.data_ptr(), 0, each.data_ptr(), 64, 1e-5)), (norm(None, one), (None, 0, one.data_ptr(), 0, 1e-5)),
                    (norm(torch.ones((4, 64)), None), None)):
        kv.append(q, k, k.clone(), slots, norm=n)
        assert calls[-1][0] == "fc_gguf_kv_append_norm" and (want is None or calls[-1][1][at] == want)
    kv.append(None, k, k.clone(), slots, norm=norm(each, one))     # without queries their weights are not looked at
    assert calls[-1][1][at] == (None, 0, one.data_ptr(), 0, 1e-5)
    kv.append(q, k, k.clone(), slots)
    assert calls[-1][0] == "fc_gguf_kv_append"
    n = len(calls)
    for bad in (norm(each, one), norm(one, torch.ones((4, 64))), norm(torch.ones(96), None), norm(torch.ones((4, 96)), None),
                norm(torch.ones((1, 4, 64)), None)):
        with pytest.raises(ValueError):
            kv.append(q, k, k.clone(), slots, norm=bad)
    assert len(calls) == n


def test_oracle_codes():
    table = o8.e4m3_values()
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(table, want, equal_nan=True)
    # every value, the middles between neighbours (ties to the even code) and just beside them
    fine = np.sort(np.unique(table[np.isfinite(table)]))
    assert np.array_equal(o8.nearest(fine), fine)
    for a, b in zip(fine[:-1], fine[1:]):
        mid = (a + b) / 2
        assert o8.nearest(mid * (1 + 1e-9 * np.sign(mid)) if mid else 1e-9) in (a, b)
        even = min((x for x in (a, b)), key=lambda x: int(np.flatnonzero(table == x)[0]) & 1)
        assert o8.nearest(mid) == even


def test_oracle_scales():
    # 448 is the largest code: 2^0; a little more: 2^1; the bounds
    for dtype, low, high in (("float16", -14, 8), ("bfloat16", -110, 120)):
        for amax, e in ((448.0, 0), (448.1, 1), (1.75, -8), (1.7501, -7), (0.0, low), (2.0 ** -130, low)):
            got = o8.quantise(np.array([[amax, -amax / 3]]), dtype)[1][0]
            assert got == max(low, e), (dtype, amax, got)
        y, e = o8.quantise(np.array([[240 * 2.0 ** high + 2.0 ** high, np.nan, np.inf, 1.0]]), dtype)
        assert e[0] == high and y[0, 0] == 240 and np.isnan(y[0, 1]) and np.isnan(y[0, 2])
    codes, scales = np.zeros((1, 1, 2, 16, 8), np.uint8), np.full((1, 1, 16), 127, np.uint8)
    codes[0, 0, 0, 3, 1], scales[0, 0, 3] = 0x38, 130
    assert o8.held(codes, scales, "float16", False)[0, 0, 0, 3, 1] == 8.0
    codes = np.zeros((1, 1, 2, 16, 8), np.uint8)
    codes[0, 0, 1, 5, 2], scales[0, 0, 10] = 0x38, 124
    assert o8.held(codes, scales, "float16", True)[0, 0, 1, 5, 2] == 0.125


def test_oracle_norm():
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(o8.head_norm(x, np.array([1.0, 2.0]), 0.0), [[[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]]])
