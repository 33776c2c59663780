"""Router linear layer's backward for dense logit gradients against the fp64 oracle."""
import numpy as np
import pytest
import torch

import synthetic
from gpu_helpers import np_, require_gpu
from oracle import training

pytestmark = pytest.mark.gpu

CASES = [                       # T, H, E
    (1, 128, 1),                # one token, one expert
    (1, 4096, 8),
    (256, 128, 4),              # tiny layer
    (4096, 4096, 8),            # Mixtral router
    (2048, 2048, 64),           # fine-grained
    (127, 384, 5),
    (129, 256, 16),
    (1025, 640, 17),
    (777, 128, 100),
    (300, 896, 255),
    (1000, 1024, 256),
    (20011, 256, 9),
]


def _inputs(T, H, E, seed=0):
    x = synthetic.random_bf16((T, H), 11 + seed)
    w = synthetic.random_bf16((E, H), 12 + seed, std=0.02)
    dx0 = synthetic.random_bf16((T, H), 13 + seed, std=1e-3)
    rng = np.random.default_rng(100 * E + T + seed)
    g = (rng.standard_normal((T, E)) * 1e-3).astype(np.float32)
    g += (rng.random((T, E)) < 2 / E) * rng.standard_normal((T, E)).astype(np.float32) * 0.02
    return x, w, dx0, g.astype(np.float32)


def _check(dx, dw, x, w, dx0, g):
    T, E = g.shape
    X, W, G = x.double().numpy(), w.double().numpy(), g.astype(np.float64)
    D = None if dx0 is None else dx0.double().numpy()
    rdx, rdw = training.router_linear_bwd(X, W, G, D)
    # dx: one bf16 rounding (2^-8), the gradients in two bf16 parts (2^-16) and a sum over the experts
    S = np.abs(G) @ np.abs(W) + (0 if D is None else np.abs(D))
    bound = 2.0 ** -8 * np.abs(rdx) + (2.0 ** -16 + (E + 8) * 2.0 ** -23) * S
    assert (np.abs(np_(dx) - rdx) <= bound + 1e-37).all()
    # dW: fp32 sums over chunks of at most 256 tokens, then over the chunks
    S = np.abs(G).T @ np.abs(X)
    assert (np.abs(np_(dw) - rdw) <= (300 + T / 64) * 2.0 ** -23 * S + 1e-37).all()
    # errors of single roundings do not line up: 2^-24 sqrt(300), with a margin
    assert np.linalg.norm(np_(dw) - rdw) <= 2e-6 * np.linalg.norm(rdw) + 1e-30


@pytest.mark.parametrize("with_dx", [True, False])
@pytest.mark.parametrize("T,H,E", CASES)
def test_router_linear_bwd(T, H, E, with_dx):
    m = require_gpu()
    x, w, dx0, g = _inputs(T, H, E)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = m.mxg_router_linear_bwd(x.cuda(), w.cuda(), torch.from_numpy(g).cuda(), dx0.cuda() if with_dx else None,
                                     status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _check(dx, dw, x, w, dx0 if with_dx else None, g)


@pytest.mark.parametrize("T,H,E", [(12000, 2048, 8), (9000, 1024, 64)])
def test_many_tiles_per_sm(T, H, E):
    """Every SM goes round its buffers several times; the second call repeats the first bit for bit."""
    m = require_gpu()
    x, w, dx0, g = _inputs(T, H, E)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd, wd, gd, dd = x.cuda(), w.cuda(), torch.from_numpy(g).cuda(), dx0.cuda()
    dx, dw = m.mxg_router_linear_bwd(xd, wd, gd, dd, status)
    for _ in range(20):
        dx2, dw2 = m.mxg_router_linear_bwd(xd, wd, gd, dd, status)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    assert int(status.item()) == 0
    _check(dx, dw, x, w, dx0, g)


@pytest.mark.parametrize("with_dx", [True, False])
@pytest.mark.parametrize("T,H,E", [
    (30000, 128, 100),          # one tile of columns: new tokens at every tile
    (20001, 256, 256),          # two, all groups' gradients replaced after them
    (12000, 640, 150),          # three groups, an odd number of tiles of columns
    (9001, 1024, 70),           # two groups, of which the second is nearly empty
])
def test_groups_of_experts_over_many_tiles(T, H, E, with_dx):
    """More than 64 experts: their gradients stay while an SM goes along the columns, and are replaced at the end."""
    m = require_gpu()
    x, w, dx0, g = _inputs(T, H, E)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd, wd, gd, dd = x.cuda(), w.cuda(), torch.from_numpy(g).cuda(), dx0.cuda() if with_dx else None
    dx, dw = m.mxg_router_linear_bwd(xd, wd, gd, dd, status)
    for _ in range(10):
        dx2, dw2 = m.mxg_router_linear_bwd(xd, wd, gd, dd, status)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    assert int(status.item()) == 0
    _check(dx, dw, x, w, dx0 if with_dx else None, g)


def test_in_place_repeatable_and_on_another_stream():
    m = require_gpu()
    x, w, dx0, g = _inputs(3001, 512, 12)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd, wd, gd, buf = x.cuda(), w.cuda(), torch.from_numpy(g).cuda(), dx0.cuda()
    a, dwa = m.mxg_router_linear_bwd(xd, wd, gd, dx0.cuda(), status)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b, dwb = m.mxg_router_linear_bwd(xd, wd, gd, buf, status, dx=buf, stream=s)
    s.synchronize()
    assert b.data_ptr() == buf.data_ptr()
    assert torch.equal(a, b) and torch.equal(dwa, dwb)
    _check(b, dwb, x, w, dx0, g)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e6, 1e30])
def test_gradients_of_any_size(scale):
    """The gradients' split into bf16 parts keeps fp32's range."""
    m = require_gpu()
    x, w, _, g = _inputs(200, 256, 8)
    g = (g * np.float32(scale)).astype(np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = m.mxg_router_linear_bwd(x.cuda(), w.cuda(), torch.from_numpy(g).cuda(), None, status)
    torch.cuda.synchronize()
    _check(dx, dw, x, w, None, g)


def test_agrees_with_the_sparse_backward():
    """On gradients that are zero off the chosen experts it is mxg_router_bwd's result."""
    m = require_gpu()
    T, H, E, k = 500, 512, 16, 3
    x, w, dx0, _ = _inputs(T, H, E)
    rng = np.random.default_rng(3)
    z = rng.standard_normal((T, E)).astype(np.float32)
    ids, probs = m.mxg_route_topk(torch.from_numpy(z).cuda(), k)
    dprobs = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sparse_dx = dx0.cuda()
    sparse_dw = m.mxg_router_bwd(x.cuda(), w.cuda(), ids, probs, dprobs, sparse_dx, status)
    g = m.mxg_balance_loss_bwd(torch.from_numpy(z).cuda(), torch.zeros(E, dtype=torch.int32, device="cuda"),
                               torch.zeros(1, dtype=torch.int32, device="cuda"), k, 1.0, status,
                               route=(ids, probs, dprobs))
    dx, dw = m.mxg_router_linear_bwd(x.cuda(), w.cuda(), g, dx0.cuda(), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    a, b = np_(dx), np_(sparse_dx)
    # both are one bf16 rounding from the exact sum
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 1e-6).all()
    assert np.linalg.norm(np_(dw) - np_(sparse_dw)) <= 4e-6 * np.linalg.norm(np_(sparse_dw))
