"""Pins of the serving operators' CPU oracle: closed forms and identities."""

import numpy as np

from oracle import serving as o


def test_rotation_by_hand():
    # a quarter turn: (x0, x1) -> (-x1, x0); both orders of pairs, a passing tail, two axes
    f = np.array([np.pi / 2, np.pi / 2])
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y, mag = o.rotate(x, [[1]], f)
    assert np.allclose(y[0, 0], [-3, -4, 1, 2, 5]) and np.allclose(mag[0, 0], [4, 6, 4, 6, 0])
    y, _ = o.rotate(x, [[1]], f, interleaved=True)
    assert np.allclose(y[0, 0], [-2, 1, -4, 3, 5])
    y, _ = o.rotate(x, [[1], [0]], f, axis=[0, 1])
    assert np.allclose(y[0, 0], [-3, 2, 1, 4, 5])
    y, _ = o.rotate(x, [[1]], f, scale=2.0)
    assert np.allclose(y[0, 0], [-6, -8, 2, 4, 5])


def test_rotation_depends_on_differences_of_positions():
    g = np.random.default_rng(1)
    q, k = g.normal(size=(2, 1, 1, 8))
    f = 10.0 ** -np.arange(4)
    dots = [(o.rotate(q, [[p + 3]], f)[0] * o.rotate(k, [[p]], f)[0]).sum() for p in (0, 11, 1000)]
    assert np.allclose(dots, dots[0])


def _pages(K, V, order, ps, pages):
    """Keys and values [n, hk, D] laid out token by token on the pages `order`."""
    n, hk, D = K.shape
    kp, vp = np.full((pages, hk, D // 8, ps, 8), np.nan), np.full((pages, hk, ps // 8, D, 8), np.nan)
    for j in range(n):
        for h in range(hk):
            for d in range(D):
                kp[order[j // ps], h, d // 8, j % ps, d % 8] = K[j, h, d]
                vp[order[j // ps], h, j % ps // 8, d, j % 8] = V[j, h, d]
    return kp, vp


def test_slots_and_attention_against_a_dense_softmax():
    g = np.random.default_rng(2)
    n, hk, D, ps = 37, 2, 16, 16
    K, V = g.normal(size=(2, n, hk, D))
    order = [4, 0, 2]
    kp, vp = _pages(K, V, order, ps, 5)
    for j in (0, 15, 16, 36):
        s = order[j // ps] * ps + j % ps
        assert np.array_equal(o.key_slot(kp, s), K[j]) and np.array_equal(o.value_slot(vp, s), V[j])
    q = g.normal(size=(3, 4, D))
    r = o.attend(q, kp, vp, [0, 3], [n], np.array([order]), 0.5, window=9)
    for i in range(3):
        for h in range(4):
            at = slice(n - 3 + i - 8, n - 3 + i + 1)
            z = 0.5 * K[at, h // 2] @ q[i, h]
            w = np.exp(z) / np.exp(z).sum()
            assert np.allclose(r["out"][i, h], w @ V[at, h // 2]) and np.isclose(r["lse"][i, h], np.log(np.exp(z).sum()))
    # joining two halves by their lse gives the whole
    a = o.attend(q, kp, vp, [0, 3], [n], np.array([[4, -1, -1]]), 0.5)
    b = o.attend(q, kp, vp, [0, 3], [n], np.array([[-1, 0, 2]]), 0.5)
    c = o.attend(q, kp, vp, [0, 3], [n], np.array([order]), 0.5)
    wa, wb = np.exp(a["lse"] - c["lse"])[..., None], np.exp(b["lse"] - c["lse"])[..., None]
    assert np.allclose(a["out"] * wa + b["out"] * wb, c["out"])


def test_rows_that_see_nothing():
    kp, vp = np.zeros((1, 1, 2, 16, 8)), np.zeros((1, 1, 2, 16, 8))
    r = o.attend(np.ones((3, 1, 16)), kp, vp, [0, 1, 3], [0, 1], np.array([[0], [0]]), 1.0)
    assert (r["out"][:2] == 0).all() and (r["lse"][:2] == -np.inf).all() and r["lse"][2, 0] == 0


def test_logits_by_hand():
    x = [[2.0, -2.0, 1.0, 4.0]]
    y, _ = o.logits(x, tokens=[[0, 1, 1, 3, 9]], lens=[3], prompt_lens=[1], repetition=[2.0], frequency=[0.5],
                    presence=[0.25], bias=[[(2, 1.0), (2, 0.5), (7, 1.0)]], mask=[[0b0111]])
    assert np.array_equal(y, [[1.0, -4.0 - 1.0 - 0.25, 2.5, -np.inf]])
