"""The oracle of the choice of the next token at random numbers of 1 and more, which count as 1 - 2^-52."""

import math

import pytest

from oracle import sampling as o


@pytest.mark.parametrize("u", [1.0, 1.5, math.inf])
def test_numbers_of_one_and_more(u):
    # a last token with a share past 2^-52 (2.2e-16) is the last, one with less is not: e^-30 is 9e-14, e^-40 4e-18
    for row, want in (([0.0, -30.0], 1), ([0.0, -40.0], 0), ([0.0, -100.0], 0), ([-100.0, 0.0], 1), ([2.0, 2.0], 1)):
        assert o.choose(row, u)[0] == want
    assert o.choose([3.0, 2.0, 1.0], u, top_k=2)[0] == 1 and o.choose([3.0, 2.0, 1.0], u)[0] == 2


def test_numbers_below_one():
    for u in (-1.0, math.nan, 0.0):
        assert o.choose([0.0, 1.0], u)[0] == 1
    assert o.choose([0.0, 1.0], 1 - 2.0 ** -24)[0] == 0
