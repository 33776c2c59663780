"""The training example: router, balance loss, experts, dense router backward and the weights' update together."""
import os
import sys

import numpy as np
import pytest
import torch

import synthetic
from conftest import ROOT
from gpu_helpers import np_, require_gpu
from oracle import training

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_example_learns_and_repeats():
    require_gpu()
    import train_moe_layer
    a = train_moe_layer.train(steps=40)
    assert torch.isfinite(a).all()
    assert a[-5:, 0].mean() < 0.8 * a[:5, 0].mean()          # the error falls
    # the balance loss is coef for a uniform router and grows with any expert's share
    assert (a[:, 1] >= 0.05 * 0.99).all() and a[-5:, 2].mean() < 0.25
    b = train_moe_layer.train(steps=40)
    assert torch.equal(a, b)                                  # every kernel's sums have a fixed order


def test_balance_gradient_through_the_router_weights():
    """d loss / d W_r and d loss / d x through both kernels, along random directions, against central differences of
    the fp64 loss (the route and so the counts held fixed)."""
    m = require_gpu()
    T, H, E, k, coef = 64, 128, 6, 2, 1.0
    x, w = synthetic.random_bf16((T, H), 41), synthetic.random_bf16((E, H), 42, std=0.05)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    logits, ids, _ = m.mxg_router_fwd(x.cuda(), w.cuda(), k)
    _, counts, _, n = m.mxg_balance_loss_fwd(logits, ids, coef, status)
    dlogits = m.mxg_balance_loss_bwd(logits, counts, n, k, coef, status)
    dx, dw = m.mxg_router_linear_bwd(x.cuda(), w.cuda(), dlogits, None, status)
    torch.cuda.synchronize()
    X, W, I = x.double().numpy(), w.double().numpy(), np_(ids).astype(np.int64)

    def loss(X, W):
        return training.balance_loss(X @ W.T, I, coef)[0]

    rng = np.random.default_rng(43)
    for grad, at in ((np_(dw).astype(np.float64), "w"), (np_(dx).astype(np.float64), "x")):
        for _ in range(4):
            d = rng.standard_normal(grad.shape)
            h = 1e-4
            if at == "w":
                num = (loss(X, W + h * d) - loss(X, W - h * d)) / (2 * h)
            else:
                num = (loss(X + h * d, W) - loss(X - h * d, W)) / (2 * h)
            # dx is rounded to bf16 (2^-9 of each element, errors that do not line up); dw is fp32; the differences
            # are off by h^2 times the third derivative
            tol = (2.0 ** -9 if at == "x" else 1e-5) * 6 * np.linalg.norm(grad * d) + 1e-6 * np.linalg.norm(grad)
            assert abs(num - (grad * d).sum()) <= tol, at
