"""Pins of the attention oracle: hand-worked values, invariants, differences and brute force (CPU)."""
import math

import numpy as np
import pytest

import oracle


def rng(seed):
    return np.random.default_rng(seed)


def test_norm_of_a_hand_worked_row():
    # x = (3, 4, 0, 0): mean square 25/4, so x / rms = (1.2, 1.6, 0, 0); w = (0, 1, 0, 0) doubles channel 1
    y = oracle.attn_prep(np.array([[[3.0, 4.0, 0.0, 0.0]]]), np.array([0.0, 1.0, 0.0, 0.0]), [7], [], eps=0.0)
    np.testing.assert_allclose(y[0, 0], [1.2, 3.2, 0.0, 0.0], rtol=1e-14)


def test_rotation_of_a_quarter_turn():
    # position 1 at pi/2 per position: (n0, n2) -> (-n2, n0); channels 1 and 3 at frequency 0 stay
    x = np.array([[[1.0, 1.0, -1.0, 1.0]]])
    y = oracle.attn_prep(x, np.zeros(4), [1], [math.pi / 2, 0.0], eps=0.0)
    np.testing.assert_allclose(y[0, 0], [1.0, 1.0, 1.0, 1.0], atol=1e-14)


def test_scores_depend_on_the_distance_alone():
    r = rng(0)
    q, k, f = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8)), [1.0, 0.1, 0.01]
    dots = [np.sum(oracle.attn_prep(q, np.zeros(8), [a], f) * oracle.attn_prep(k, np.zeros(8), [b], f))
            for a, b in ((5, 2), (105, 102), (3, 0))]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-12)


@pytest.mark.parametrize("rot", [0, 2, 6, 8])
def test_gradients_against_differences(rot):
    r = rng(rot)
    x, w, dy = r.normal(size=(3, 2, 8)), r.normal(size=8) * 0.3, r.normal(size=(3, 2, 8))
    pos, f = np.array([0, 3, 11]), 0.7 ** np.arange(rot // 2)
    dx, dw = oracle.attn_prep_backward(dy, x, w, pos, f, eps=1e-3)
    loss = lambda x, w: np.sum(dy * oracle.attn_prep(x, w, pos, f, eps=1e-3))  # noqa: E731
    h = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-8
    for i in range(8):
        e = np.zeros(8)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-8


def test_attention_against_brute_force():
    r = rng(2)
    lens, ps = [0, 1, 5, 8], 4
    k, v = r.normal(size=(6, 2, ps, 3)), r.normal(size=(6, 2, ps, 3))
    table = np.array([[0, 0], [4, 0], [1, 3], [2, 5]])
    q = r.normal(size=(4, 4, 3))
    y = oracle.attn_decode(q, k, v, table, lens, scale=0.5)
    for b in range(4):
        for h in range(4):
            num, den = np.zeros(3), 0.0
            for p in range(lens[b]):
                page = table[b, p // ps]
                e = math.exp(0.5 * sum(q[b, h, i] * k[page, h // 2, p % ps, i] for i in range(3)))
                num += e * v[page, h // 2, p % ps]
                den += e
            np.testing.assert_allclose(y[b, h], num / den if den else 0.0, rtol=1e-12)


def test_attention_over_listed_pages_is_attention_over_their_keys():
    r = rng(3)
    k, v, q = r.normal(size=(4, 1, 2, 3)), r.normal(size=(4, 1, 2, 3)), r.normal(size=(1, 2, 3))
    table, lens = np.array([[3, 1, 0]]), [5]
    y = oracle.attn_decode(q, k, v, table, lens, pages=np.array([[[0, 2, -1]]]))
    keys, values = np.stack([k[3, 0, 0], k[3, 0, 1], k[0, 0, 0]]), np.stack([v[3, 0, 0], v[3, 0, 1], v[0, 0, 0]])
    s = np.exp(q[0] @ keys.T / math.sqrt(3))
    np.testing.assert_allclose(y[0], s @ values / s.sum(1, keepdims=True), rtol=1e-12)
    assert not oracle.attn_decode(q, k, v, table, lens, pages=np.array([[[-1, -1, -1]]])).any()
    full = oracle.attn_decode(q, k, v, table, lens, pages=np.array([[[2, 0, 1]]]))
    np.testing.assert_allclose(full, oracle.attn_decode(q, k, v, table, lens), rtol=1e-12)


def test_mean_of_a_partial_page_and_of_untouched_ones():
    k = np.arange(3 * 1 * 4 * 2, dtype=float).reshape(3, 1, 4, 2)
    mean = np.full((3, 1, 2), -7.0)
    got = oracle.page_mean(k, np.array([[2, 0]]), [6], mean, [5])
    np.testing.assert_array_equal(got[0, 0], [1.0, 2.0])  # keys 0 and 1 of page 0: positions 4 and 5
    assert (got[1:] == -7).all() and (mean == -7).all()
    got = oracle.page_mean(k, np.array([[2, 0]]), [6], mean)
    np.testing.assert_array_equal(got[2, 0], k[2, 0].mean(0))


def test_choice_keeps_the_ends_and_breaks_ties_downwards():
    mean = np.zeros((6, 1, 1))
    mean[:, 0, 0] = [0.0, 5.0, 1.0, 5.0, 5.0, -9.0]
    table, q = np.arange(6)[None], np.ones((1, 1, 1))
    pick = lambda n, first, last, length=24: oracle.attn_select(q, mean, table, [length], 4, n, first, last)[0, 0].tolist()  # noqa: E731
    assert pick(2, 0, 0) == [1, 3]
    assert pick(3, 0, 1) == [1, 3, 5]
    assert pick(4, 1, 1) == [0, 1, 3, 5]
    assert pick(3, 0, 1, 7) == [0, 1, -1]  # two pages in all
    assert pick(2, 0, 1, 0) == [-1, -1]
    q2 = np.array([[[1.0], [-1.0]]])  # the second head of the group wants page 5
    assert oracle.attn_select(q2, mean, table, [24], 4, 2, 0, 0)[0, 0].tolist() == [1, 5]
