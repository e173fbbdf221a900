"""Pins of the streaming-attention oracle: facts that the mathematics fixes, and planted mistakes
that break them."""
import numpy as np
import pytest
import torch

from oracle import streaming_oracle as S


def _draw(n, d, seed, m=4):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal((n, d)) for _ in range(m)]


@pytest.mark.parametrize("n,window,sinks,causal", [(1, 1, 0, True), (9, 3, 2, True), (9, 3, 0, False), (9, 2, 12, False),
                                                   (7, 20, 0, True), (7, 1, 0, False), (8, 3, 6, False)])
def test_visibility_pair_by_pair(n, window, sinks, causal):
    m = S.visible(np.arange(n), n, window, sinks, causal)
    for i in range(n):
        for j in range(n):
            if causal:
                want = j <= i and (i - j < window or j < sinks)
            else:
                want = abs(i - j) < window or j < sinks
            assert m[i, j] == want, (i, j)


@pytest.mark.parametrize("causal", [True, False])
def test_a_window_over_everything_is_full_attention(causal):
    Q, K, V, _ = _draw(13, 8, 0)
    O, lse, _ = S.window_head(Q, K, V, 13, 0, causal, 0.3)
    q, k, v = (torch.from_numpy(x)[None, None] for x in (Q, K, V))
    ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=causal, scale=0.3)[0, 0].numpy()
    assert np.abs(O - ref).max() < 1e-13


def test_a_window_of_one_returns_the_values():
    Q, K, V, _ = _draw(6, 4, 1)
    for causal in (True, False):
        assert np.array_equal(S.window_head(Q, K, V, 1, 0, causal, 1.0)[0], V)


def test_a_row_that_sees_nothing_is_zero():
    Q, K, V, _ = _draw(3, 4, 2)
    P, lse = S.weights(Q, K, np.array([[True, False, True], [False] * 3, [True] * 3]), 1.0)
    assert not P[1].any() and lse[1] == -np.inf and np.isclose(P[[0, 2]].sum(1), 1).all()


def _finite_differences(f, x, e=1e-6):
    g = np.zeros_like(x)
    for at in np.ndindex(*x.shape):
        keep = x[at]
        x[at] = keep + e
        hi = f()
        x[at] = keep - e
        lo = f()
        x[at] = keep
        g[at] = (hi - lo) / (2 * e)
    return g


@pytest.mark.parametrize("n,window,sinks,causal", [(7, 3, 2, True), (6, 2, 1, False), (5, 9, 0, True)])
def test_gradients_against_finite_differences(n, window, sinks, causal):
    Q, K, V, dO = _draw(n, 4, 3)
    f = lambda: float((S.window_head(Q, K, V, window, sinks, causal, 0.7)[0] * dO).sum())
    got = S.window_head_backward(Q, K, V, dO, window, sinks, causal, 0.7)
    for x, g in zip((Q, K, V), got):
        assert np.abs(g - _finite_differences(f, x)).max() < 1e-8


@pytest.mark.parametrize("mistake", ["window", "sinks", "delta"])
def test_planted_mistakes_break_the_gradient(mistake):
    Q, K, V, dO = _draw(7, 4, 4)
    good = S.window_head_backward(Q, K, V, dO, 3, 1, True, 0.7)
    if mistake == "delta":
        P = S.window_head(Q, K, V, 3, 1, True, 0.7)[2]
        bad = (P * (dO @ V.T) * 0.7) @ K
    else:
        bad = S.window_head_backward(Q, K, V, dO, 4 if mistake == "window" else 3, 0 if mistake == "sinks" else 1,
                                     True, 0.7)[0]
    assert np.abs(bad - good[0]).max() > 1e-3


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_adds_angles(interleaved):
    x = np.random.default_rng(5).standard_normal(16)
    a, b = np.array([0.3, 1.1, -2.0]), np.array([0.5, -0.2, 0.9])
    r = lambda v, t: S.rotate(v, np.cos(t), np.sin(t), interleaved, torch.float64)
    y = r(x, a)
    assert np.array_equal(y[6:], x[6:].astype(np.float32))      # elements behind rope_dim stay
    assert abs(np.linalg.norm(y) - np.linalg.norm(x)) < 1e-6
    assert np.abs(r(y, b) - r(x, a + b)).max() < 1e-6
    one = r(np.eye(16)[0], np.array([np.pi / 2, 0, 0]))          # the first element's partner
    assert abs(one[1 if interleaved else 3] - 1) < 1e-7


def test_append_keeps_values_within_half_a_step():
    rng = np.random.default_rng(6)
    rows = rng.standard_normal((16, 8)) * np.geomspace(0.1, 10, 16)[:, None]
    codes, scale = np.zeros((16, 8), np.int8), np.float32(0)
    steps = 0.0
    for t in range(16):                      # one token at a time, the scale growing on the way
        codes, new = S.append_rows(codes, scale, t, rows[t:t + 1])
        steps += 0.5 * float(new) if new > scale else 0.0        # each rescaling rounds once more
        scale = new
        assert np.abs(codes[:t + 1] * np.float64(scale) - rows[:t + 1]).max() <= steps + 0.5 * float(scale) + 1e-6
    once, s1 = S.append_rows(np.zeros((16, 8), np.int8), 0, 0, rows)
    assert s1 == scale and np.abs(once * np.float64(s1) - rows).max() <= 0.5 * float(s1) * (1 + 1e-6)


def test_append_forgets_a_page_that_starts_anew():
    codes, scale = S.append_rows(np.full((16, 4), 99, np.int8), 50.0, 0, np.full((2, 4), 1.27))
    assert scale == np.float32(np.float32(1.27) / np.float32(127)) and (codes[:2] == 127).all() and (codes[2:] == 99).all()


def test_append_of_what_is_not_finite_marks_the_page():
    for bad in (np.nan, np.inf):
        assert np.isnan(S.append_rows(np.zeros((16, 4), np.int8), 1.0, 3, np.array([[1, 2, bad, 0.]]))[1])
    assert np.isnan(S.append_rows(np.zeros((16, 4), np.int8), np.nan, 3, np.ones((1, 4)))[1])
    assert S.append_rows(np.zeros((16, 4), np.int8), np.nan, 0, np.zeros((1, 4)))[1] == 0
