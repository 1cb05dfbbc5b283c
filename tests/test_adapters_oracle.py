"""CPU pins of the adapters' oracle: hand-written values, and every gradient against
differences of the forward function."""
import numpy as np
import pytest

from oracle import adapters_oracle as AO


def rng(seed):
    return np.random.default_rng(seed)


def test_lora_add_by_hand():
    """Two adapters of rank 1, one row without an adapter, one id out of range."""
    A = np.array([[[1.0, 2.0]], [[0.0, -1.0]]])
    B = np.array([[[3.0], [4.0], [0.0]], [[1.0], [1.0], [2.0]]])
    X = np.array([[1.0, 1.0], [2.0, 3.0], [5.0, 5.0], [7.0, 7.0]])
    base = np.ones((4, 3))
    Y = AO.lora_add(X, A, B, [0, 1, -1, 2], scale=[2.0, 0.5], base=base)
    # row 0: t = 3, Y = 1 + 2 * 3 * (3, 4, 0); row 1: t = -3, Y = 1 - 1.5 * (1, 1, 2)
    assert np.array_equal(Y, [[19, 25, 1], [-0.5, -0.5, -2], [1, 1, 1], [1, 1, 1]])


def differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[i] = h
        g[i] = (f(x + d) - f(x - d)) / (2 * h)
    return g


def test_lora_gradients_against_differences():
    r = rng(1)
    M, K, N, rank, L = 7, 4, 5, 2, 3
    ids = np.array([0, 2, 0, -1, 2, 2, 5])       # adapter 1 unused, one row none, one out of range
    X, A, B = r.standard_normal((M, K)), r.standard_normal((L, rank, K)), r.standard_normal((L, N, rank))
    dY, scale = r.standard_normal((M, N)), np.array([0.5, 1.0, 2.0])
    dX, dA, dB = AO.lora_grad(dY, X, A, B, ids, scale)
    loss = lambda X, A, B: float((AO.lora_add(X, A, B, ids, scale) * dY).sum())  # noqa: E731
    # the loss is at most cubic in each argument's entries and linear in any one of them, so
    # the central difference has no truncation error: 2^-53 |loss| / h < 1e-10
    assert np.abs(dX - differences(lambda v: loss(v, A, B), X)).max() < 1e-8
    assert np.abs(dA - differences(lambda v: loss(X, v, B), A)).max() < 1e-8
    assert np.abs(dB - differences(lambda v: loss(X, A, v), B)).max() < 1e-8
    assert not dA[1].any() and not dB[1].any() and not dX[3].any() and not dX[6].any()


def test_grouped_by_hand_and_gradients_against_differences():
    r = rng(2)
    K, N, E = 3, 4, 4
    off = np.array([0, 2, 2, 5, 6])              # expert 1 empty, row 6 of no expert
    X, W, b = r.standard_normal((7, K)), r.standard_normal((E, N, K)), r.standard_normal((E, N))
    Y = AO.grouped_mm(X, off, W, b)
    for row, e in ((0, 0), (1, 0), (2, 2), (4, 2), (5, 3)):
        assert np.allclose(Y[row], W[e] @ X[row] + b[e], rtol=1e-14)
    assert not Y[6].any()
    dY = r.standard_normal((7, N))
    dX, dW, db = AO.grouped_mm_grad(dY, X, off, W)
    loss = lambda X, W, b: float((AO.grouped_mm(X, off, W, b) * dY).sum())  # noqa: E731
    assert np.abs(dX - differences(lambda v: loss(v, W, b), X)).max() < 1e-8
    assert np.abs(dW - differences(lambda v: loss(X, v, b), W)).max() < 1e-8
    assert np.abs(db - differences(lambda v: loss(X, W, v), b)).max() < 1e-8


@pytest.mark.parametrize("planted", ["scale", "rows", "transpose"])
def test_planted_mistake_is_caught(planted):
    """A wrong gradient (scale dropped, a row of another adapter, A and B exchanged) differs
    from the differences by far more than their error."""
    r = rng(3)
    X, A, B = r.standard_normal((3, 2)), r.standard_normal((2, 2, 2)), r.standard_normal((2, 2, 2))
    dY, ids, scale = r.standard_normal((3, 2)), np.array([0, 1, 0]), np.array([0.5, 3.0])
    right = differences(lambda v: float((AO.lora_add(X, v, B, ids, scale) * dY).sum()), A)
    if planted == "scale":
        wrong = AO.lora_grad(dY, X, A, B, ids, None)[1]
    elif planted == "rows":
        wrong = AO.lora_grad(dY, X, A, B, np.array([0, 0, 0]), scale)[1]
    else:
        wrong = AO.lora_grad(dY, X, A, B.transpose(0, 2, 1), ids, scale)[1]
    assert np.abs(wrong - right).max() > 1e-2
