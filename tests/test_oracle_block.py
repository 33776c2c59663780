"""The oracle of the block operators against differences and hand-made cases (no GPU needed)."""
import numpy as np
import pytest

from oracle import block


def test_rms_norm_gradient_is_the_difference():
    rng = np.random.default_rng(0)
    T, H, eps = 3, 7, 1e-3
    r, w, dy, dres = (rng.standard_normal(s) for s in ((T, H), (H,), (T, H), (T, H)))

    def loss(r, w):
        return (block.rms_norm(r, w, eps)[2] * dy).sum() + (r * dres).sum()

    d, dw = block.rms_norm_grad(dy, r, w, block.rms_norm(r, w, eps)[1], dres)
    h = 1e-6
    for i in range(T):
        for j in range(H):
            e = np.zeros_like(r)
            e[i, j] = h
            assert abs((loss(r + e, w) - loss(r - e, w)) / (2 * h) - d[i, j]) < 1e-7
    for j in range(H):
        e = np.zeros_like(w)
        e[j] = h
        assert abs((loss(r, w + e) - loss(r, w - e)) / (2 * h) - dw[j]) < 1e-7


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_is_the_difference(kind, renormalize):
    rng = np.random.default_rng(1)
    T, E, k = 4, 9, 3
    z, dp = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    ids, p = block.route(z, k, kind, renormalize=renormalize, scale=2.5)
    d = block.route_grad(z, ids, p, dp, kind, renormalize, 2.5)

    def loss(z):                                       # the choice held fixed
        w = np.take_along_axis(block.scores(z, kind), ids, axis=1)
        return (2.5 * (w / w.sum(axis=1, keepdims=True) if renormalize else w) * dp).sum()

    h = 1e-6
    for i in range(T):
        for j in range(E):
            e = np.zeros_like(z)
            e[i, j] = h
            assert abs((loss(z + e) - loss(z - e)) / (2 * h) - d[i, j]) < 1e-7


def test_route_choices():
    z = np.array([[0.0, 1.0, 2.0, 3.0, 2.5, -np.inf, 0.0, 0.0]])
    assert block.route(z, 3, "softmax")[0].tolist() == [[3, 4, 2]]
    # the bias chooses, the weights stay the scores'
    ids, w = block.route(z, 2, "sigmoid", bias=np.array([5, 0, 0, 0, 0, 9, 0, 0.0]), renormalize=False)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, [[0.5, 1 / (1 + np.exp(-3))]])
    # groups of two: sums of scores 1.23, 1.83, 0.92 (one is off), 1.0: the first two
    ids, _ = block.route(z, 4, "sigmoid", groups=4, top_groups=2, group_top=2)
    assert ids.tolist() == [[3, 2, 1, 0]]
    # by their largest the third stays instead, with its expert that is off last
    ids, w = block.route(z, 4, "sigmoid", groups=4, top_groups=2, group_top=1)
    assert ids.tolist() == [[3, 4, 2, 5]] and w[0, 3] == 0.0
    ids, w = block.route(np.full((1, 4), -np.inf), 2, "softmax")
    assert ids.tolist() == [[0, 1]] and not w.any()


def test_grad_norm_of_any_size():
    for scale in (1e-40, 1e-3, 1e30):
        assert abs(block.grad_norm([np.array([3.0 * scale]), np.array([4.0 * scale, 0.0])]) / (5 * scale) - 1) < 1e-12
    assert block.grad_norm([np.zeros(3)]) == 0.0
