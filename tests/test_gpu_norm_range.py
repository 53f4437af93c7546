"""Head norms of bf16 over the whole range of the type: the squares of its largest and smallest values are not f32's.

The tolerances are those of test_gpu_kv8.py: the bound of a norm in f32 is relative, so it holds for heads of any size.
Where eps outweighs a small head its results fall below bf16's normal range, whose step there is 2^-133: such a rounding
is off by half of that, 2^-134, whatever the value, and by 2^-140 at most come the few f32 operations (steps of 2^-149)
before it.
"""

import numpy as np
import pytest
import torch

from oracle import serving as o
from oracle import serving8 as o8
from test_gpu_kv8 import BF16, F32, _before, _check_append, _half, _i32, _kv8, _np, _randn, _slots

pytestmark = pytest.mark.gpu

# powers of two of a head's values: below bf16's normal range to its largest, with the borders of f32's squares between
POWERS = (-132, -120, -100, -76, -70, -64, -63, -62, -40, -1, 0, 20, 60, 61, 62, 63, 64, 65, 100, 123, 125)


def _heads(tg, T, heads, D, shift):
    """Heads of random values, each about a power of two of its own, cut at the type's largest."""
    by = torch.tensor([[2.0 ** POWERS[(t + shift + 5 * h) % len(POWERS)] for h in range(heads)] for t in range(T)], dtype=torch.float64)
    x = torch.randn((T, heads, D), generator=tg).double() * by[..., None]
    top = torch.finfo(BF16).max
    return x.clamp(-top, top).to(BF16).cuda()


def _cache(bits, pages, ps, hk, D):
    from gguf_quant_block_amd.serving import PagedKv
    if bits == 8:
        return _kv8(pages, ps, hk, D, BF16)
    kv = PagedKv(pages, ps, hk, D, BF16)
    kv.k.fill_(7.0)
    kv.v.fill_(7.0)
    return kv


def _near(y, x, w, eps, pos, f):
    """Whether y are the normed and rotated heads x."""
    D = x.shape[-1]
    want, mag = o8.head_norm(_np(x), _np(w), eps), 0.0
    if f is not None:
        want, mag = o.rotate(want, pos, f, None, False, 1.0)
    err = 2.0 ** -21 * mag + (D / 2 + 8) * 2.0 ** -24 * np.where(mag > 0, mag, np.abs(want))
    tol = err + _half(BF16) * (np.abs(want) + err) + 2.0 ** -134 + 2.0 ** -140
    assert (np.abs(y - want) <= tol).all(), float((np.abs(y - want) - tol).max())


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-34])
def test_large_and_small_heads(gpu_lib, D, bits, eps):
    from gguf_quant_block_amd.serving import HeadNorm, Rope
    T, hq, hk, ps = 2 * len(POWERS) + 1, 3, 2, 16
    g, tg = np.random.default_rng(D), torch.Generator().manual_seed(D)
    slots, pages = _slots("prompt", T, ps, g)
    q, k, v = _heads(tg, T, hq, D, 0), _heads(tg, T, hk, D, 2), _randn(tg, (T, hk, D), BF16)
    w = [torch.rand((n, D), generator=tg).add(0.5).cuda() for n in (hq, hk)]
    f = torch.tensor([10000.0 ** (-2 * j / 64) for j in range(32)], dtype=F32, device="cuda")
    pos = g.integers(0, 200000, (1, T))
    for rope in (None, Rope(f)):
        kv = _cache(bits, pages, ps, hk, D)
        before = _before(kv)
        norm = HeadNorm(*w, eps=eps)
        out = kv.append(q, k, v, _i32(slots), _i32(pos[0]) if rope else None, rope, norm=norm)
        turn = (pos, _np(f)) if rope else (None, None)
        _near(_np(out), q, w[0], eps, *turn)
        if bits == 8:                                            # (codes' steps are 2^-120 at least)
            _check_append(kv, before, k, k, v, slots, *turn, False, 1.0, norm, None)
        else:
            held = _np(kv.k)
            _near(np.stack([o.key_slot(held, s) for s in slots]), k, w[1], eps, *turn)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_ordinary_heads_beside_them_keep_their_bits(gpu_lib, D):
    from gguf_quant_block_amd.serving import HeadNorm
    T, hq, hk = 8, 6, 2
    tg = torch.Generator().manual_seed(D)
    q, k = (_randn(tg, (T, h, D), BF16) for h in (hq, hk))
    norm = HeadNorm(_randn(tg, (D,), F32), _randn(tg, (D,), F32), eps=1e-5)
    outs = []
    for x in (None, 2.0 ** 100, 2.0 ** -120, float("inf"), float("nan")):
        z = q.clone()
        if x is not None:
            z[:, ::2, :D // 2] = x
        kv = _cache(16, 2, 16, hk, D)
        outs.append((kv.append(z, k, k, _i32(range(T)), norm=norm), kv.k[0, :, :, :T].clone()))
    for out, keys in outs[1:]:
        assert torch.equal(out[:, 1::2], outs[0][0][:, 1::2]) and torch.equal(keys, outs[0][1])
    # an infinite value: itself over itself, and the others over it
    out = outs[3][0][:, ::2]
    assert torch.isnan(out[..., :D // 2]).all() and (out[..., D // 2:] == 0).all()
    assert torch.isnan(outs[4][0][:, ::2]).all()
