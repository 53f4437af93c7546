"""Attention with one dominant key (a sink) among many of small weights: together these hold mass that the output must
not lose.  The weights are rounded to the cache's type for the second product; an f16 weight is off by 2^-11 of itself,
or, below 2^-14 in the units of the product, by 2^-25 there.  The units put a row's largest weight at 2^8 or more, so
that a weight is off by 2^-33 of the largest at most: 2^-33 of the values' sum in the tolerance, 2^-8 of what the other
tests leave."""

import numpy as np
import pytest
import torch

from test_gpu_attend_paths import _reference
from test_gpu_serving import BF16, F16, _half, _i32, _kv, _layout, _np

pytestmark = pytest.mark.gpu


# (D, page, kv heads, group, keys, new tokens): shares of the streaming kernel (one and two row tiles), a sequence that
# is not split, tiles of 128 rows, split tiles, tiles of 256 rows
@pytest.mark.parametrize("D,ps,hk,G,kv_len,new", [(64, 16, 2, 4, 20000, 1), (128, 64, 1, 8, 9000, 4), (256, 32, 1, 2, 9000, 1),
                                                  (96, 16, 3, 1, 1000, 1), (128, 16, 2, 2, 2500, 90), (64, 64, 1, 4, 9000, 40),
                                                  (256, 16, 1, 1, 3000, 70), (96, 32, 2, 2, 3000, 60), (64, 16, 64, 4, 900, 256),
                                                  (128, 64, 64, 4, 900, 256)])
@pytest.mark.parametrize("where", ["first", "middle", "late"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_weights_beside_a_sink(gpu_lib, dtype, where, D, ps, hk, G, kv_len, new):
    g, tg = np.random.default_rng(kv_len), torch.Generator().manual_seed(kv_len)
    table, pages = _layout([kv_len], ps, g)
    kv = _kv(pages, ps, hk, D, dtype, fill=0.0)
    # scores in powers of two: 0 for the sink, -23 .. -27 for the others
    level = torch.from_numpy(-23.0 - 4.0 * g.random(kv_len))
    level[{"first": 0, "middle": kv_len // 2, "late": kv_len - new}[where]] = 0.0
    key = torch.arange(kv_len)
    page = torch.from_numpy(np.repeat(table[0], ps)[:kv_len].copy()).long()
    kv.k[page.cuda(), :, 0, (key % ps).cuda(), 0] = level.to(dtype).cuda()[:, None]
    values = (1.0 + 0.25 * torch.randn((kv_len, hk, D), generator=tg)).to(dtype).cuda()
    values[level == 0.0] = 0.0
    kv.v[page.cuda(), :, (key % ps // 8).cuda(), :, (key % 8).cuda()] = values
    q = torch.zeros((new, hk * G, D), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    out, lse = torch.empty_like(q), torch.empty((new, hk * G), device="cuda")
    cu, scale = [0, new], float(np.log(2.0))
    kv.attend(q, _i32(cu), _i32([kv_len]), _i32(table), new, scale=scale, out=out, lse=lse)
    r = _reference(q, kv, cu, [kv_len], table, scale, 0)
    half, want = _half(dtype), r["out"]
    # a score is one product of at most 27 ln 2 and sums of zeros: off by 2^-22 of it (the product and the factor log2(e))
    weight = 2 * 2.0 ** -22 * r["score"][..., None] + 2.0 ** -21 + (r["keys"][..., None] + 64) * 2.0 ** -23
    tol = r["mass"] * (1.01 * half + weight) + half * np.abs(want)
    if dtype == F16:
        tol = tol + 2.0 ** -25 + 2.0 ** -33 * r["vsum"]
    err = np.abs(_np(out) - want)
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.2f} tolerances, {float((err / want).max()):.3f} of the value"
    tl = 2.0 ** -22 * r["score"] + 2.0 ** -20 + (r["keys"] + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(r["lse"])
    assert (np.abs(_np(lse) - r["lse"]) <= tl).all()
