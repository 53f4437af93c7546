"""Calls of unusual lengths: a long chunk beside hundreds of single tokens, and row offsets that are not in order."""

import numpy as np
import pytest
import torch

from helpers import guarded
from oracle import serving as o
from test_gpu_attend_paths import _case
from test_gpu_serving import BF16, F16, F32, _fill, _i32, _kv, _layout, _near_attend, _np

pytestmark = pytest.mark.gpu


# rows of the chunk times the sequences, over all key heads, are more than a grid of every sequence's longest could hold
@pytest.mark.parametrize("dtype,D,hk,G,chunk,seqs,window", [(F16, 64, 32, 16, 512, 512, 0), (BF16, 128, 16, 8, 700, 1500, 50)])
def test_chunk_beside_many_single_tokens(gpu_lib, dtype, D, hk, G, chunk, seqs, window):
    g = np.random.default_rng(seqs)
    kvs = [chunk + 100] + g.integers(1, 60, seqs - 1).tolist()
    news = [chunk] + [1] * (seqs - 1)
    at = seqs // 3                                  # among the others
    kvs[0], kvs[at] = kvs[at], kvs[0]
    news[0], news[at] = news[at], news[0]
    _case(dtype, D, 16, hk, G, kvs, news, window=window, seed=seqs)


@pytest.mark.parametrize("new", [6, 60])
@pytest.mark.parametrize("cu", [[-3, 400, 2], [5, 3, 400], [400, 500, 600], [-9, -5, 7], [0, 2**31 - 1, -2**31]])
def test_offsets_out_of_order_or_range(gpu_lib, cu, new):
    """Offsets are clamped to the rows of q and never go back; nothing else is read or written."""
    T, kvs = 2 * new, [64, 70]
    g, tg = np.random.default_rng(5), torch.Generator().manual_seed(5)
    table, pages = _layout(kvs, 16, g)
    kv = _kv(pages, 16, 1, 64, F16)
    _fill(kv, table, kvs, tg)
    q = torch.randn((T, 4, 64), generator=tg).half().cuda()
    out, guard = guarded((T, 4, 64), F16, seed=1)
    lse, lse_guard = guarded((T, 4), F32, seed=2)
    out.fill_(9.0)
    lse.fill_(9.0)
    kv.attend(q, _i32(cu), _i32(kvs), _i32(table), new, out=out, lse=lse)
    guard()
    lse_guard()
    got, got_lse, written = _np(out), _np(lse), np.zeros(T, bool)
    for s in range(2):
        a = min(max(cu[s], 0), T)
        b = min(max(cu[s + 1], a), T)
        r = o.attend(_np(q)[a:b], _np(kv.k), _np(kv.v), [0, b - a], kvs[s:s + 1], table[s:s + 1], 0.125, max_q=new)
        n = min(b - a, new)
        if n:
            _near_attend(got[a:a + n], got_lse[a:a + n], {k: x[:n] for k, x in r.items()}, F16, 64)
        assert not written[a:a + n].any()
        written[a:a + n] = True
    assert (got[~written] == 9).all() and (got_lse[~written] == 9).all()
