"""The float64 oracle of the layer operators against facts that fix it: rotations keep
lengths and undo themselves, scores depend on position differences only, the gradient
agrees with differences, and activations with their limits."""
import math

import numpy as np
import pytest

from oracle import layer_oracle as lo

ROPES = {
    "three-axes": lo.rope((8, 4, 4), (2, 3, 4)),
    "half": lo.rope((6, 6, 4), (3, 2, 4), style="half", start=(5, 0, 0)),
    "one-axis-partial": lo.rope((10,), (24,), theta=500.0),
    "two-axes-text": lo.rope((8, 8), (3, 5), first=4, scale=(0.5, 2.0)),
}


@pytest.mark.parametrize("name", list(ROPES))
def test_rotation_keeps_lengths_and_inverts(name):
    x = np.random.default_rng(0).standard_normal((2, 3, 24, 16))
    r = ROPES[name]
    y = lo.rotate(x, r)
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-12)
    assert np.allclose(lo.rotate(y, r, inverse=True), x, atol=1e-12)


def test_scores_depend_on_position_differences():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    r = lo.rope((8, 4, 4), (40, 40, 40))

    def score(a, b):
        qa = lo.rotate(q, r, np.array(a).reshape(1, 1, 3))
        kb = lo.rotate(k, r, np.array(b).reshape(1, 1, 3))
        return float((qa * kb).sum())

    assert math.isclose(score((3, 4, 5), (1, 1, 1)), score((23, 14, 35), (21, 11, 31)), rel_tol=1e-12)
    assert not math.isclose(score((3, 4, 5), (1, 1, 1)), score((4, 4, 5), (1, 1, 1)), rel_tol=1e-6)


def test_first_position_and_text_do_not_turn():
    x = np.random.default_rng(2).standard_normal((1, 1, 24, 16))
    y = lo.rotate(x, ROPES["two-axes-text"])
    assert np.array_equal(y[:, :, :5], x[:, :, :5]) and np.array_equal(y[:, :, 19:], x[:, :, 19:])
    assert not np.allclose(y[:, :, 5:19], x[:, :, 5:19])


@pytest.mark.parametrize("name", list(ROPES))
def test_gradient_agrees_with_differences(name):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 1, 2, 24, 16))
    w = 1 + 0.2 * rng.standard_normal(16)
    r, eps, h = ROPES[name], 1e-3, 1e-6
    dx, dw = lo.norm_rotate_grad(x, w, eps, dy, r)

    def loss(x_, w_):
        return float((lo.norm_rotate(x_, w_, eps, r) * dy).sum())

    for at in [(0, 0, 0, 0), (0, 1, 7, 5), (0, 1, 23, 15)]:
        e = np.zeros_like(x)
        e[at] = h
        # central differences: error h^2 and rounding 1e-16 / h, both under 1e-7 here
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for i in (0, 9):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_activations():
    z = np.array([-40.0, -1.0, 0.0, 1.0, 40.0])
    for act in ("gelu_tanh", "gelu_erf", "silu"):
        y = lo.activate(z, act)
        assert abs(y[0]) < 1e-15 and y[2] == 0 and y[4] == 40.0
    assert math.isclose(lo.activate(np.array([1.0]), "gelu_erf")[0], 0.8413447460685429, rel_tol=1e-12)
    assert math.isclose(lo.activate(np.array([1.0]), "silu")[0], 1 / (1 + math.exp(-1)), rel_tol=1e-12)


def test_linear_head_major_equals_token_major():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 3, 5, 8))
    w, gate, res = rng.standard_normal((7, 24)), rng.standard_normal((2, 7)), rng.standard_normal((2, 5, 7))
    a, _ = lo.linear(x, w, None, gate, res, "silu")
    b, _ = lo.linear(x.transpose(0, 2, 1, 3).reshape(2, 5, 24), w, None, gate, res, "silu")
    assert np.allclose(a, b, atol=1e-14)
