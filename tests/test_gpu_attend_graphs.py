"""Captured attention beside eager calls of other sizes on the same handle: the graph's workspace stays, and the replays
give the eager call's bits."""

import numpy as np
import pytest
import torch

from oracle import serving as o
from test_gpu_serving import F16, _fill, _i32, _kv, _layout, _near_attend, _np, _randn

pytestmark = pytest.mark.gpu


def _capture(call):
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        call()
    torch.cuda.synchronize()
    return graph


class _Step:
    """Attention of the last `new` tokens of a sequence of `keys`."""

    def __init__(self, kv, table, tg, keys, new, heads):
        self.kv, self.keys, self.new, self.table = kv, keys, new, table
        self.q = _randn(tg, (new, heads, kv.head_dim), kv.dtype)
        self.args = (_i32([0, new]), _i32([keys]), _i32(table), new)
        self.out, self.lse = torch.empty_like(self.q), torch.empty((new, heads), device="cuda")

    def __call__(self):
        self.kv.attend(self.q, *self.args, out=self.out, lse=self.lse)

    def check(self):
        r = o.attend(_np(self.q), _np(self.kv.k), _np(self.kv.v), [0, self.new], [self.keys], self.table, self.kv.scale)
        _near_attend(_np(self.out), _np(self.lse), r, self.kv.dtype, self.kv.head_dim)


@pytest.mark.parametrize("largest_first", [True, False])
def test_replays_after_calls_of_other_sizes(gpu_lib, largest_first):
    g, tg = np.random.default_rng(21), torch.Generator().manual_seed(21)
    keys, heads = 4000, 64
    table, pages = _layout([keys], 16, g)
    kv = _kv(pages, 16, 8, 64, F16)
    _fill(kv, table, [keys], tg)
    # the tiles of 1100 tokens fill the CUs unsplit and take no workspace, those of 64 are split
    step, middle, large = (_Step(kv, table, tg, keys, new, heads) for new in (1, 64, 1100))
    if largest_first:
        large()
    else:
        step()
    graph = _capture(step)
    step()
    want = [t.clone() for t in (step.out, step.lse)]
    step.check()
    for other in (middle, large, middle, step):
        other()
        if other is middle:
            other.check()
        for _ in range(2):
            step.out.fill_(float("nan"))
            step.lse.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(step.out, want[0]) and torch.equal(step.lse, want[1])
    # a second graph, of a size whose call came after the first graph
    again = _capture(middle)
    middle()
    want2 = middle.out.clone()
    for _ in range(3):
        graph.replay()
        again.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out, want[0]) and torch.equal(middle.out, want2)


def test_first_call_in_a_capture_where_nothing_is_split(gpu_lib):
    g, tg = np.random.default_rng(22), torch.Generator().manual_seed(22)
    table, pages = _layout([500], 16, g)
    kv = _kv(pages, 16, 2, 64, F16)
    _fill(kv, table, [500], tg)
    step = _Step(kv, table, tg, 500, 1, 8)
    graph = _capture(step)
    for _ in range(3):
        step.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        step.check()
