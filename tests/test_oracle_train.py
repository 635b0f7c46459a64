"""The 64-bit training-step operators against their definitions: closed forms,
splitting over ranks, and gradients against central differences."""

import numpy as np
import pytest

from oracle import train as O


def _rng(k):
    return np.random.default_rng([7, k])


def test_cross_entropy_of_equal_logits_is_log_vocab():
    x, ws = np.ones((3, 4)), [np.zeros((5, 4)), np.zeros((6, 4))]
    loss, lse = O.cross_entropy(x, ws, np.array([0, 10, -1]))
    assert np.allclose(lse, np.log(11)) and np.allclose(loss, [np.log(11), np.log(11), 0.0])


def test_cross_entropy_does_not_depend_on_the_split():
    r = _rng(1)
    x, w, y = r.normal(size=(5, 8)), r.normal(size=(13, 8)), np.array([0, 12, 5, 13, -4])
    whole, parts = O.cross_entropy(x, [w], y), O.cross_entropy(x, [w[:4], w[4:4], w[4:]], y)
    assert all(np.allclose(a, b) for a, b in zip(whole, parts))
    assert np.array_equal(whole[0][3:], [0.0, 0.0])


def test_cross_entropy_gradient_against_differences():
    r = _rng(2)
    x, ws, y = r.normal(size=(4, 6)), [r.normal(size=(3, 6)), r.normal(size=(5, 6))], np.array([7, -1, 0, 3])
    d = r.normal(size=4)
    _, lse = O.cross_entropy(x, ws, y)
    dx, dw = O.cross_entropy_grad(x, ws, y, lse, d)
    total = lambda: float((O.cross_entropy(x, ws, y)[0] * d).sum())  # noqa: E731
    for a, da in ((x, dx), (ws[0], dw[0]), (ws[1], dw[1])):
        for i in np.ndindex(a.shape):
            keep, h = a[i], 1e-6
            a[i] = keep + h
            up = total()
            a[i] = keep - h
            down = total()
            a[i] = keep
            assert abs((up - down) / (2 * h) - da[i]) < 1e-7
    assert not dx[1].any()


def test_balance_loss_of_a_uniform_router():
    # every expert chosen equally often with equal probabilities: coef * E * E * (1/E)(1/E) = coef
    z, idx = [np.zeros((4, 4))] * 2, [np.arange(4)[:, None].astype(np.int32)] * 2
    counts, loss, grads = O.balance_loss(z, idx, 0.5)
    assert counts.tolist() == [[1] * 4, [1] * 4, [2] * 4] and abs(loss - 0.5) < 1e-15
    assert not np.array(grads).any()


def test_balance_gradient_against_differences():
    r = _rng(3)
    z = [r.normal(size=(3, 5)), r.normal(size=(0, 5)), r.normal(size=(4, 5))]
    idx = [np.array([[0, 4], [-1, -1], [2, 9]], np.int32), np.zeros((0, 2), np.int32),
           np.array([[1, 2], [1, 1], [-1, 3], [0, 4]], np.int32)]
    counts, _, grads = O.balance_loss(z, idx, 0.7)
    assert counts[-1].tolist() == [2, 3, 2, 1, 2] and not grads[0][1].any()
    for a, da in zip(z, grads):
        for i in np.ndindex(a.shape):
            keep, h = a[i], 1e-6
            a[i] = keep + h
            up = O.balance_loss(z, idx, 0.7)[1]
            a[i] = keep - h
            down = O.balance_loss(z, idx, 0.7)[1]
            a[i] = keep
            assert abs((up - down) / (2 * h) - da[i]) < 1e-8


@pytest.mark.parametrize("shape", [(6, 6), (4, 9), (9, 4), (1, 5)])
def test_orthogonalize_acts_on_singular_values(shape):
    g = _rng(4).normal(size=shape)
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + 1e-7)
    for a, b, c in [O.DEFAULT_COEFFS] * 4:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(O.orthogonalize(g, 4), (u * s) @ v, atol=1e-9)


def test_orthogonalize_cubic_converges_to_the_polar_factor():
    g = _rng(5).normal(size=(5, 8))
    u, _, v = np.linalg.svd(g, full_matrices=False)
    assert np.allclose(O.orthogonalize(g, 16, [(1.5, -0.5, 0.0)] * 16), u @ v, atol=1e-6)
    assert not O.orthogonalize(np.zeros((3, 4)), 5).any()
