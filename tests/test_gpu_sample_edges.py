"""Sampling at the ends of its settings, where the definition alone says what the result is."""

import math

import pytest
import torch

from oracle import sampling as o

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


def test_numbers_of_one_and_more(gpu_lib):
    """They count as 1 - 2^-52: a last token that holds less of the sum than 2^-52 is not chosen, and one that weighs less
    than 2^-64 of the largest never is."""
    from gguf_quant_block_amd.serving import sample
    rows = [[0.0, -30.0], [0.0, -40.0], [0.0, -100.0], [2.0, 2.0], [-100.0, 0.0], [1.0, -math.inf], [0.0, -1e30]]
    want = [1, 0, 0, 1, 1, 0, 0]
    for v in (1.0, 1.5, math.inf):
        out = sample(_f32(rows), _f32([v] * len(rows)))
        assert out.tolist() == want
        assert [o.choose(r, v)[0] for r in rows] == want
    # rows of many tokens, which are taken apart by bins; the last of equal ones is the last id
    x = torch.zeros((2, 20000), device="cuda")
    x[1, :10000] = -100.0
    for v in (1.0, 7.0):
        assert sample(x, _f32([v, v])).tolist() == [19999, 19999]
    x[1] = 0
    x[1, 15000:] = -100.0
    assert sample(x, _f32([1.0, 1.0])).tolist() == [19999, 14999]
    # the kept tokens end before: the last of them
    x = torch.arange(20000, device="cuda").flip(0).float()[None] / 20000
    for k in (1, 7, 600, 9000):
        assert sample(x, _f32([1.0]), top_k=torch.tensor([k], dtype=torch.int32, device="cuda")).tolist() == [k - 1]
