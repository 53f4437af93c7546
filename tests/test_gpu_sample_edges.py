"""Sampling at the ends of its settings, where the definition alone says what the result is."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _f32(x):
    return torch.tensor(x, dtype=F32, device="cuda")


@pytest.mark.parametrize("vocab", [5, 300, 20000, 131073])
@pytest.mark.parametrize("min_p", [1.0, 0.999999940395, 0.5, 1e-30])
def test_infinite_temperature(gpu_lib, vocab, min_p):
    """exp((x - top) / inf) is 1 for every finite logit: all weigh the same, and all of them at least min_p."""
    from gguf_quant_block_amd.serving import sample
    tg = torch.Generator().manual_seed(vocab)
    # logits that all differ, so that the order of the tokens is known
    x = (torch.randperm(vocab, generator=tg).float() / 64 - 3).repeat(4, 1)
    hidden = vocab // 4
    x[:, torch.randperm(vocab, generator=tg)[:hidden]] = -math.inf
    n = vocab - hidden
    order = x[0].argsort(descending=True)[:n]
    ranks = [0, n // 3, n // 2, n - 1]
    u = [(r + 0.5) / n for r in ranks]                          # the middles of these tokens' shares
    lp = torch.empty(4, device="cuda")
    out = sample(x.cuda(), _f32(u), temperature=_f32([math.inf] * 4), min_p=_f32([min_p] * 4), logprobs=lp)
    assert out.tolist() == order[ranks].tolist()
    # a sum of n equal whole numbers is exact; its logarithm is rounded to f64, within 2^-50 with the division, and to f32
    assert all(abs(y + math.log(n)) <= (2.0 ** -24 + 2.0 ** -50) * math.log(n) for y in lp.tolist())


def test_infinite_temperature_beside_ends_of_min_p(gpu_lib):
    from gguf_quant_block_amd.serving import sample
    x = _f32([[1.0, 0.0, -1.0]] * 3)
    inf = math.inf
    # min_p past 1 leaves the first; a finite temperature leaves what weighs as much as the first
    out = sample(x, _f32([0.9] * 3), temperature=_f32([inf, 1.0, inf]), min_p=_f32([1.5, 1.0, 0.0]))
    assert out.tolist() == [0, 0, 2]
    x[:, 1] = inf                                                # an infinite logit leaves only its like, at any temperature
    assert sample(x, _f32([0.9] * 3), temperature=_f32([inf] * 3), min_p=_f32([1.0, 0.5, 0.0])).tolist() == [1, 1, 1]
