"""The training operators' oracle pinned against differences and closed forms (CPU)."""
import numpy as np
import pytest

from oracle import training


def _case(T, E, k, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) * 1.5
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    return z, ids, rng


@pytest.mark.parametrize("T,E,k,masked", [(7, 4, 2, False), (5, 9, 3, True), (1, 3, 1, False)])
def test_balance_grad_against_differences(T, E, k, masked):
    z, ids, rng = _case(T, E, k, 1)
    mask = rng.random(T) < 0.6 if masked else None
    _, counts, _, n = training.balance_loss(z, ids, 0.3, mask)
    g = training.balance_grad(z, counts, n, k, 0.3, 1.7, mask)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            zp, zm = z.copy(), z.copy()
            zp[t, e] += h
            zm[t, e] -= h
            num = 1.7 * (training.balance_loss(zp, ids, 0.3, mask)[0] - training.balance_loss(zm, ids, 0.3, mask)[0]) / (2 * h)
            # central differences: error O(h^2) + rounding 1e-16 / h
            assert abs(num - g[t, e]) < 1e-9


def test_balance_loss_of_uniform_router_is_coef():
    T, E, k = 12, 4, 2
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    loss, counts, sums, n = training.balance_loss(np.zeros((T, E)), ids, 0.25)
    assert abs(loss - 0.25) < 1e-15 and n == T
    assert (counts == T * k // E).all() and np.allclose(sums, T / E)


def test_balance_empty_rows():
    z, ids, _ = _case(6, 5, 2, 2)
    z[2] = -np.inf
    assert not training.softmax_rows(z)[2].any()
    loss, counts, _, n = training.balance_loss(z, ids, 1.0, np.zeros(6, bool))
    assert loss == 0.0 and n == 0 and not counts.any()
    assert not training.balance_grad(z, counts, 0, 2, 1.0).any()


def test_route_grad_against_differences():
    z, ids, rng = _case(6, 7, 3, 3)
    dprobs = rng.standard_normal((6, 3))

    def value(zz):
        c = np.take_along_axis(zz, ids, axis=1)
        e = np.exp(c - c.max(axis=1, keepdims=True))
        return float(((e / e.sum(axis=1, keepdims=True)) * dprobs).sum())

    c = np.take_along_axis(z, ids, axis=1)
    e = np.exp(c - c.max(axis=1, keepdims=True))
    g = training.route_grad(ids, e / e.sum(axis=1, keepdims=True), dprobs, 7)
    h = 1e-5
    for t in range(6):
        for i in range(7):
            zp, zm = z.copy(), z.copy()
            zp[t, i] += h
            zm[t, i] -= h
            assert abs((value(zp) - value(zm)) / (2 * h) - g[t, i]) < 1e-8


def test_router_linear_bwd_against_differences():
    rng = np.random.default_rng(4)
    x, w, g = rng.standard_normal((5, 6)), rng.standard_normal((3, 6)), rng.standard_normal((5, 3))
    dx, dw = training.router_linear_bwd(x, w, g)
    h = 1e-4
    for a, d in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + h
            up = float((g * (x @ w.T)).sum())
            a[i] = old - h
            dn = float((g * (x @ w.T)).sum())
            a[i] = old
            assert abs((up - dn) / (2 * h) - d[i]) < 1e-9


@pytest.mark.parametrize("m,n", [(5, 9), (9, 5), (6, 6), (1, 4), (4, 1)])
def test_orthogonalise_maps_the_singular_values(m, n):
    """X keeps its singular vectors; each singular value goes through the scalar polynomial."""
    rng = np.random.default_rng(5)
    u = rng.standard_normal((m, n))
    a, b, c = co = (3.4445, -4.7750, 2.0315)
    P, s, Q = np.linalg.svd(u, full_matrices=False)
    s = s / np.sqrt((s * s).sum())
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(training.orthogonalise(u, 5, co), (P * s) @ Q, atol=1e-12)


def test_orthogonalise_zero_and_momentum():
    assert not training.orthogonalise(np.zeros((3, 4)), 5, (3.4445, -4.775, 2.0315)).any()
    g, m = np.ones((2, 2)), np.full((2, 2), 2.0)
    new, u = training.momentum(g, m, 0.5, True)
    assert (new == 2.0).all() and (u == 2.0).all()
    new, u = training.momentum(g, m, 0.5, False)
    assert (u == new).all()
