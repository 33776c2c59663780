"""Balance loss of the router and its gradient on the GPU against the fp64
oracle, within bounds on the fp32 arithmetic, and against differences."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import training

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CASES = [                       # T, E, k, masked, disabled experts
    (1, 1, 1, False, 0),        # one token, one expert
    (1, 8, 2, False, 0),
    (2, 2, 2, True, 0),
    (77, 5, 1, False, 0),       # rows of odd length
    (256, 4, 2, True, 0),       # tiny layer
    (4096, 8, 2, False, 0),     # Mixtral router
    (1001, 9, 3, True, 1),      # one past eight experts
    (999, 17, 4, True, 2),
    (8192, 64, 8, False, 0),    # fine-grained layer
    (3001, 60, 4, True, 5),
    (130, 129, 8, False, 1),
    (700, 256, 32, True, 7),    # the widest route
    (40000, 33, 3, True, 0),    # several tokens per lane group
]


def _inputs(T, E, k, masked, disabled, seed=0):
    rng = np.random.default_rng(1000 * E + T + seed)
    z = (rng.standard_normal((T, E)) * 2.0 + rng.standard_normal((1, E))).astype(np.float32)
    if disabled:
        z[:, rng.choice(E, min(disabled, E - k), replace=False)] = -np.inf
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = rng.random(T) < 0.8 if masked else None
    return z, ids, mask, rng


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _spread(z):
    """Largest distance of a finite logit from its row's maximum: exp's argument, whose rounding is relative to it."""
    d = z.max(axis=1, keepdims=True) - z
    return float(d[np.isfinite(d)].max(initial=0.0))


def _p_rel(z):
    # z - top rounds once (spread * U), expf is within 2 ulp (4 U), the sum of up to 256 terms is 8 in a row
    # and 5 by halves, then a reciprocal and a product
    return (_spread(z) + 4 + 13 + 3) * U


@pytest.mark.parametrize("T,E,k,masked,disabled", CASES)
def test_balance_fwd(T, E, k, masked, disabled):
    m = require_gpu()
    z, ids, mask, _ = _inputs(T, E, k, masked, disabled)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, counts, sums, n = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 0.01, status, token_mask=_dev(mask))
    torch.cuda.synchronize()
    rl, rc, rs, rn = training.balance_loss(z, ids, 0.01, mask)
    assert int(status.item()) == 0
    assert int(n.item()) == rn
    assert np.array_equal(np_(counts), rc)
    # sums of non-negative terms: each partial is a chain of at most T / 32 additions per lane, then
    # 5 + 8 + (up to 152 blocks)
    rel = _p_rel(z) + (T / 32 + 5 + 8 + 152) * U
    assert (np.abs(np_(sums) - rs) <= rel * rs + 1e-37).all()
    assert abs(float(loss.item()) - rl) <= (rel + 20 * U) * rl


@pytest.mark.parametrize("route", [False, True])
@pytest.mark.parametrize("T,E,k,masked,disabled", CASES)
def test_balance_bwd(T, E, k, masked, disabled, route):
    m = require_gpu()
    z, ids, mask, rng = _inputs(T, E, k, masked, disabled)
    _, counts, _, n = training.balance_loss(z, ids, 0.01, mask)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = dq = None
    if route:
        c = np.take_along_axis(z.astype(np.float64), ids, axis=1)
        e = np.exp(c - c.max(axis=1, keepdims=True))
        q = (e / e.sum(axis=1, keepdims=True)).astype(np.float32)
        dq = (rng.standard_normal((T, k)) * 0.01 / T).astype(np.float32)
    got = m.mxg_balance_loss_bwd(_dev(z), _dev(counts.astype(np.int32)), torch.full((1,), n, dtype=torch.int32, device="cuda"),
                                 k, 0.01, status, dloss=torch.full((1,), 0.75, device="cuda"), token_mask=_dev(mask),
                                 route=(_dev(ids), _dev(q), _dev(dq)) if route else None)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref = training.balance_grad(z, counts, n, k, 0.01, 0.75, mask)
    live = np.ones(T, bool) if mask is None else mask
    p = training.softmax_rows(np.where(live[:, None], z, -np.inf))
    dev = (E * counts.astype(np.float64) - k * n) / max(k * n, 1)
    # (d_e - sum p d) E / ...: each p within _p_rel, the deviations within 2 U, a sum of 13 steps, 4 products
    bound = 0.75 * 0.01 / max(n, 1) * p * (np.abs(dev)[None, :] + (p @ np.abs(dev))[:, None]) * (_p_rel(z) + 24 * U)
    if route:
        ref = ref + training.route_grad(ids, q, dq, E)
        inner = np.abs(q * dq).astype(np.float64).sum(axis=1, keepdims=True)
        b = np.abs(q) * (np.abs(dq) * 4 + (k + 8) * inner) * U
        full = np.zeros((T, E))
        np.put_along_axis(full, ids.astype(np.int64), b, axis=1)
        bound = bound + full + U * np.abs(ref)
    assert (np.abs(np_(got) - ref) <= bound + 1e-37).all()


def test_gradient_is_the_losses_difference():
    """The GPU gradient against central differences of the fp64 loss."""
    m = require_gpu()
    T, E, k, coef = 24, 6, 2, 0.5
    z, ids, mask, _ = _inputs(T, E, k, True, 0, 5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, counts, _, n = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), coef, status, token_mask=_dev(mask))
    g = np_(m.mxg_balance_loss_bwd(_dev(z), counts, n, k, coef, status, token_mask=_dev(mask)))
    h = 1e-4
    z64 = z.astype(np.float64)
    for t in range(T):
        for e in range(E):
            zp, zm = z64.copy(), z64.copy()
            zp[t, e] += h
            zm[t, e] -= h
            num = (training.balance_loss(zp, ids, coef, mask)[0] - training.balance_loss(zm, ids, coef, mask)[0]) / (2 * h)
            # differences: h^2 times the third derivative (below coef E / n) and 1e-16 / h; fp32: 1e-6 of coef E / n
            assert abs(num - g[t, e]) <= 2e-6 * coef * E / int(n.item())


def test_balanced_router_has_no_cancellation():
    """Counts equal up to one token: the bracket is ~1e-4 of f, and stays accurate to fp32."""
    m = require_gpu()
    T, E, k = 8192, 8, 1
    rng = np.random.default_rng(9)
    z = (rng.standard_normal((T, E)) * 0.1).astype(np.float32)
    ids = (np.arange(T) % E).astype(np.int32).reshape(T, 1)
    ids[0, 0] = 3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, counts, _, n = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 1.0, status)
    g = np_(m.mxg_balance_loss_bwd(_dev(z), counts, n, k, 1.0, status)).astype(np.float64)
    ref = training.balance_grad(z, np_(counts), T, k, 1.0)
    # with f itself in fp32 the error would be U / (1 / T) ~ 5e-4 of the result
    assert np.linalg.norm(g - ref) <= 2e-6 * np.linalg.norm(ref)


@pytest.mark.parametrize("T,E", [(9, 2), (300, 4), (4096, 32)])
def test_every_expert_chosen_has_no_gradient(T, E):
    """k = E: every f is 1 / E whatever the router does, the loss is coef and its gradient exactly zero."""
    m = require_gpu()
    z, ids, mask, _ = _inputs(T, E, E, True, 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, counts, _, n = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 0.5, status, token_mask=_dev(mask))
    g = m.mxg_balance_loss_bwd(_dev(z), counts, n, E, 0.5, status, token_mask=_dev(mask))
    assert not g.any()
    # the sums of a token's p: each within _p_rel of exact; T n-term additions in blocks and a few products
    assert abs(float(loss.item()) - 0.5) <= 0.5 * (_p_rel(z) + 100 * U)


def test_masked_and_infinite_rows():
    m = require_gpu()
    z, ids, _, _ = _inputs(64, 12, 3, False, 0)
    z[3] = -np.inf                                   # no expert open for this token
    z[5] = np.nan                                    # dropped by the mask: must not be read into anything
    z[6] = np.inf
    mask = np.ones(64, bool)
    mask[[5, 6, 9]] = False
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, counts, sums, n = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 1.0, status, token_mask=_dev(mask))
    g = np_(m.mxg_balance_loss_bwd(_dev(z), counts, n, 3, 1.0, status, token_mask=_dev(mask.astype(np.uint8))))
    rl, rc, rs, rn = training.balance_loss(z, ids, 1.0, mask)
    assert rn == int(n.item()) == 61 and np.array_equal(np_(counts), rc)
    assert abs(float(loss.item()) - rl) <= 1e-5 * rl
    assert np.isfinite(g).all() and not g[[3, 5, 6, 9]].any()
    # every token dropped
    loss, counts, sums, n = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 1.0, status, token_mask=_dev(np.zeros(64, bool)))
    g = m.mxg_balance_loss_bwd(_dev(z), counts, n, 3, 1.0, status, token_mask=_dev(np.zeros(64, bool)))
    assert float(loss.item()) == 0.0 and int(n.item()) == 0 and not counts.any() and not sums.any() and not g.any()
    # NaN that counts is not hidden
    loss, *_ = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 1.0, status)
    assert np.isnan(float(loss.item()))
    assert int(status.item()) == 0


def test_lowest_value_masks_and_large_logits():
    """Experts masked by the type's lowest value, and rows far from zero."""
    m = require_gpu()
    z, ids, _, _ = _inputs(200, 10, 2, False, 0)
    z[:, 7] = np.finfo(np.float32).min
    z[50:100] += 1e4
    z[100:150] -= 1e4
    ids = np.argsort(-z, axis=1, kind="stable")[:, :2].astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, counts, sums, _ = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 1.0, status)
    rl, rc, rs, _ = training.balance_loss(z, ids, 1.0)
    assert np.array_equal(np_(counts), rc)
    assert abs(float(loss.item()) - rl) <= 1e-5 * rl
    assert (np.abs(np_(sums) - rs) <= 1e-5 * rs).all()


def test_bad_expert_ids_are_reported():
    m = require_gpu()
    z, ids, _, _ = _inputs(100, 6, 2, False, 0)
    bad = ids.copy()
    bad[7, 1] = 6
    bad[8, 0] = -1
    for call in ("fwd", "bwd"):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if call == "fwd":
            _, counts, _, _ = m.mxg_balance_loss_fwd(_dev(z), _dev(bad), 1.0, status)
            assert np.array_equal(np_(counts), training.balance_loss(z, bad, 1.0)[1])
        else:
            one = torch.full((100, 2), 0.5, device="cuda")
            m.mxg_balance_loss_bwd(_dev(z), torch.ones(6, dtype=torch.int32, device="cuda"),
                                   torch.full((1,), 100, dtype=torch.int32, device="cuda"), 2, 1.0, status,
                                   route=(_dev(bad), one, one))
        assert int(status.item()) == 16


def test_repeatable_and_on_another_stream():
    m = require_gpu()
    z, ids, mask, _ = _inputs(30011, 60, 4, True, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zd, idd, md = _dev(z), _dev(ids), _dev(mask)
    a = m.mxg_balance_loss_fwd(zd, idd, 0.01, status, token_mask=md)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = m.mxg_balance_loss_fwd(zd, idd, 0.01, status, token_mask=md, stream=s)
    s.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
