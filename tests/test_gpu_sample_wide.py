"""Sampling of rows of more slices than a workgroup keeps in its shared memory (64), or has threads (1024), against rows
sorted in float64 and summed with 64 bits of fraction.

Tolerances as in test_gpu_sample.py: rows whose border comes within 2^-32 of the sum say nothing.  Sums of 2^23 numbers
with 64 bits of fraction are off by 2^-41 of themselves at most.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SLICE = 4096                                                     # tokens of a slice of few rows


def _choose(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (token, log of its share, margin)."""
    x = x.astype(np.float64)
    order = np.argsort(-x, kind="stable")
    order = order[:int((x > -np.inf).sum())]
    z = x[order]
    w = np.exp(((z - z[0]) / temperature).astype(np.longdouble))
    n, margin = len(w), 1.0
    if top_k > 0:
        n = min(n, top_k)
    c = np.cumsum(w[:n])
    if top_p < 1:
        least = top_p * c[-1]
        n = min(n, int(np.searchsorted(c, least)) + 1)
        margin = min(margin, float(np.abs(c - least).min() / c[-1]))
    if min_p > 0:
        margin = min(margin, float(np.abs(w[1:] / min_p - 1).min()))
        n = max(1, min(n, int((w[:n] >= min_p).sum())))
    c = c[:n]
    t = u * c[-1]
    if n > 1:
        margin = min(margin, float(np.abs(c[:-1] - t).min() / c[-1]))
    at = min(int(np.searchsorted(c, t, side="right")), n - 1)
    return int(order[at]), float(np.log(w[at] / c[-1])), margin


def _check(x, settings, us):
    from gguf_quant_block_amd.serving import sample
    rows = x.shape[0]
    z = x.double().cpu().numpy()
    unsure = 0
    for kw in settings:
        full = {k: torch.full((rows,), v, dtype=torch.int32 if k == "top_k" else F32, device="cuda") for k, v in kw.items()}
        seen = {k: v[0].item() for k, v in full.items()}         # (as rounded to f32)
        for u in us:
            ut, lp = torch.full((rows,), u, device="cuda"), torch.empty(rows, device="cuda")
            out = sample(x, ut, logprobs=lp, **full).tolist()
            for r in range(rows):
                want, share, margin = _choose(z[r], ut[r].item(), **seen)
                if margin < 2.0 ** -32:
                    unsure += 1
                    continue
                assert out[r] == want, (r, kw, u, out[r], want, margin)
                assert abs(lp[r].item() - share) <= 2.0 ** -32 + 2.0 ** -24 * abs(share), (r, kw, u)
    assert unsure <= 1, unsure


FILTERS = [{}, {"temperature": 0.7}, {"top_k": 40}, {"top_k": 5000}, {"top_p": 0.9}, {"min_p": 0.02},
           {"temperature": 1.3, "top_k": 900, "top_p": 0.95, "min_p": 0.001}]


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("spread", [0.3, 2.5, 8.0])
def test_more_than_64_slices(gpu_lib, dtype, spread):
    tg = torch.Generator().manual_seed(int(spread * 10))
    x = torch.randn((2, 300001), generator=tg) * spread
    # the first tokens on both sides of the border between slices 63 and 64, and in the last slice
    at = 64 * SLICE
    x[0, at - 40:at + 40] = spread * 4.5 + torch.randn(80, generator=tg)
    x[1, 300001 - 30:] = spread * 4.5 + torch.randn(30, generator=tg)
    x[1, :63 * SLICE] -= spread
    _check(x.to(dtype).cuda(), FILTERS, (0.0, 0.31, 0.77, 0.9999))


@pytest.mark.parametrize("rows", [1, 3, 13])
def test_stretches_of_slices_past_the_64th(gpu_lib, rows):
    """Slices that have to be read again alternate with such as need not be: stretches that begin and end on both sides
    of slice 64, whatever parts they are read in."""
    tg = torch.Generator().manual_seed(rows)
    n = 140
    x = torch.randn((rows, n * SLICE), generator=tg) * 0.8
    lift = torch.rand((rows, n), generator=tg) < 0.5
    lift[:, 60:68] = True
    lift[:, 100:] = False
    x = (x.view(rows, n, SLICE) + 3.0 * lift[..., None]).view(rows, -1)[:, 3:]      # an odd length
    x[:, -1] = 9.0
    _check(x.cuda(), [{}, {"top_k": 3000}, {"top_p": 0.4}, {"min_p": 0.01}], (0.02, 0.6))


def test_equal_logits(gpu_lib):
    x = torch.full((2, 300001), -1.25, device="cuda")
    x[1, 64 * SLICE + 5:] = -1.0
    _check(x, [{}, {"top_p": 0.7}, {"top_k": 280000}], (0.0, 0.5, 0.97))


def test_more_than_1024_slices(gpu_lib):
    tg = torch.Generator().manual_seed(4)
    vocab = 1027 * 8192 + 77
    x = torch.randn((1, vocab), generator=tg) * 2
    x[0, 1024 * 8192 - 20:1024 * 8192 + 30] = 14.0 + torch.randn(50, generator=tg)
    x[0, -3:] = 15.0
    _check(x.to(BF16).cuda(), [{}, {"top_k": 60}, {"top_p": 0.3, "min_p": 1e-4}], (0.1, 0.55, 0.98))
    # the largest in the last slice, and nothing that it outweighs is written down by the others
    x = torch.randn((1, vocab), generator=tg) * 0.5
    x[0, vocab - 9] = 18.0
    _check(x.cuda(), [{}, {"top_p": 0.9}], (0.4, 0.95))
