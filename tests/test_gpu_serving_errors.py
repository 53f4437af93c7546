"""An error that an earlier call of the runtime left behind is not the serving operators': their calls answer for
themselves, and leave it to its owner."""

import ctypes

import numpy as np
import pytest
import torch

from test_gpu_serving import F16, _i32, _kv, _np

pytestmark = pytest.mark.gpu


@pytest.fixture
def pending(gpu_lib):
    """A function that leaves an error behind (an unknown attribute asked for), and the runtime."""
    torch.zeros(1, device="cuda")
    with open("/proc/self/maps") as f:
        hip = ctypes.CDLL(next(line.split()[-1] for line in f if "libamdhip64" in line))
    value = ctypes.c_int()
    yield lambda: hip.hipDeviceGetAttribute(ctypes.byref(value), 99999, 0), hip
    hip.hipGetLastError()


def test_calls_after_an_error_of_others(pending):
    from gguf_quant_block_amd.serving import Rope, process_logits
    leave, hip = pending
    kv = _kv(400, 16, 2, 64, F16, fill=0.0)
    x = torch.full((2, 2, 64), 2.0, dtype=F16, device="cuda")
    rope, pos = Rope(torch.zeros(32, device="cuda")), _i32([5, 6])
    table = _i32(np.arange(400)[None])
    logits = torch.arange(40.0, device="cuda")[None]
    out = [torch.zeros_like(x), torch.zeros_like(x), torch.zeros((64, 2, 64), dtype=F16, device="cuda"), torch.zeros_like(logits)]
    q64 = torch.ones((64, 2, 64), dtype=F16, device="cuda")
    args = [(_i32([0, 2]), _i32([2]), _i32([[0]]), 2), (_i32([0, 64]), _i32([6400]), table, 64)]
    slots = _i32([0, 1])
    torch.cuda.synchronize()
    calls = (lambda: kv.append(x, x, x, slots, pos, rope, out=out[0]),
             lambda: kv.attend(x, *args[0], out=out[1]),              # the streaming kernel
             lambda: kv.attend(q64, *args[1], out=out[2]),            # tiles, split and joined; the workspace grows
             lambda: process_logits(logits, out=out[3]))
    for call in calls:
        assert leave() != 0
        call()
        assert hip.hipGetLastError() != 0                             # still there
    assert (_np(out[0]) == 2).all() and (_np(out[1]) == 2).all() and np.array_equal(_np(out[3]), _np(logits))
    first = out[2].clone()
    calls[2]()
    assert torch.equal(out[2], first) and (_np(first) > 0).all()
