"""Attention over 8 bits where its result is known to the bit, and the sign of infinite results."""

import numpy as np
import pytest
import torch

from oracle import serving as o
from test_gpu_kv8 import BF16, F16, _attend8_case, _held, _i32, _kv8, _layout, _near_attend, _np, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,ps,G,new,window", [(64, 16, 2, 200, 0), (96, 32, 2, 150, 0), (128, 64, 2, 130, 0), (256, 64, 1, 140, 0),
                                               (128, 16, 4, 100, 300), (64, 128, 1, 257, 33), (96, 256, 1, 140, 0), (256, 16, 2, 65, 0)])
def test_tiles_equal_those_of_16_bits(gpu_lib, dtype, D, ps, G, new, window):
    """Codes are turned into values of the type on their way to shared memory, exactly, and all that follows is the same:
    so are the bits."""
    from gguf_quant_block_amd.serving import PagedKv
    kv, q, cu, table, out, lse = _attend8_case(dtype, D, ps, 2, G, [900, 301], [new, 70], window=window, seed=new, packed=True)
    wide = PagedKv(kv.pages, ps, 2, D, dtype)
    for x, y in zip((wide.k, wide.v), _held(kv)):
        x.copy_(torch.from_numpy(y).cuda().to(dtype))
        live = np.isfinite(y)
        assert np.array_equal(_np(x)[live], y[live])
    lse16 = torch.empty_like(lse)
    other = wide.attend(q, _i32(cu), _i32([900, 301]), _i32(table), max(new, 70), window=window, lse=lse16)
    assert torch.equal(other, out) and torch.equal(lse16, lse)


@pytest.mark.parametrize("new,G", [(1, 1), (3, 4), (90, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_infinite_sums_keep_their_sign(gpu_lib, D, new, G):
    """bf16 values past 2^100 may take the f32 sums to infinity: of the sign that all values of the dimension have."""
    n, ps = 700, 32
    g, tg = np.random.default_rng(D + new), torch.Generator().manual_seed(D + new)
    table, pages = _layout([n], ps, g)
    kv = _kv8(pages, ps, 1, D, BF16)
    slots = [int(table[0][j // ps]) * ps + j % ps for j in range(n)]
    sign = torch.where(torch.rand(D, generator=tg) < 0.5, -1.0, 1.0)
    v = (torch.rand((n, 1, D), generator=tg) + 0.5) * sign * 2.0 ** 125
    kv.append(None, _randn(tg, (n, 1, D), BF16), v.to(BF16).cuda(), _i32(slots))
    q = _randn(tg, (new, G, D), BF16, 2.0)
    lse = torch.empty((new, G), device="cuda")
    got = _np(kv.attend(q, _i32([0, new]), _i32([n]), _i32(table), new, lse=lse))
    with np.errstate(over="ignore"):
        r = o.attend(_np(q), *_held(kv), [0, new], [n], table, D ** -0.5)
    assert not np.isnan(got).any()
    assert np.array_equal(np.sign(got), np.broadcast_to(sign.numpy(), got.shape))
    _near_attend(np.where(np.isinf(got), r["out"], got), _np(lse), r, BF16, D)


@pytest.mark.parametrize("dtype,D,hk,G,kvs,news", [(F16, 128, 8, 4, [4000, 31, 900, 2500], [1] * 4), (BF16, 64, 2, 4, [3001, 500], [5, 5]),
                                                   (F16, 96, 2, 2, [30000], [1]), (BF16, 256, 1, 2, [2000, 777], [90, 1]),
                                                   (BF16, 128, 2, 2, [2000, 600], [600, 600])])
def test_equal_calls_give_equal_bits(gpu_lib, dtype, D, hk, G, kvs, news):
    """Whatever else the device does and memory holds: the order of the sums goes by sizes and lengths."""
    first = None
    for i in range(4):
        junk = [torch.full((1 << 18 << i,), float("nan"), device="cuda") for _ in range(3)]
        kv, q, cu, table, out, lse = _attend8_case(dtype, D, 32, hk, G, kvs, news, seed=3)
        del junk
        for _ in range(8):                                       # (the workspace is used again)
            again, lse2 = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
            kv.attend(q, _i32(cu), _i32(kvs), _i32(table), max(news), out=again, lse=lse2)
            assert torch.equal(again, out) and torch.equal(lse2, lse)
        if first is None:
            first = out.clone(), lse.clone()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
