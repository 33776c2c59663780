"""Balance loss: the exponential over its whole range, the length of the forward's sums."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import training

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _case(T, E, k, seed):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((T, E)) * 2.0).astype(np.float32)
    return z, np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)


def test_exponential_over_its_range():
    """One token with logits 0 and -d has prob_sums 1 / s and e^-d / s, s = 1 + e^-d: their quotient is e^-d but for the
    rounding of the two products.  2^y is within 2^-22.5 < 2.83 U, the exponential rounds once more, the products
    once each: 6 U.  Below the smallest normal number (d > 87.33) the result is zero, where expf gives subnormals."""
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = np.concatenate([np.linspace(0.0, 1.0, 40), np.linspace(1.0, 87.3, 200)]).astype(np.float32)
    ids = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    sums = []
    for v in d:
        z = torch.tensor([[0.0, -float(v)]], device="cuda")
        sums.append(m.mxg_balance_loss_fwd(z, ids, 1.0, status)[2])
    s = np_(torch.stack(sums)).astype(np.float64)
    got = s[:, 1] / s[:, 0]
    ref = np.exp(-d.astype(np.float64))
    # the quotient of a product below the smallest normal number says nothing about the exponential
    ok = ref * s[:, 0] >= 2.0 ** -126
    assert ok[:-1].all()
    assert (np.abs(got - ref)[ok] <= 6 * U * ref[ok]).all()
    cuda = np_(torch.exp(-torch.from_numpy(d).cuda())).astype(np.float64)
    # expf is within 2 ulp = 4 U
    assert (np.abs(got - cuda)[ok] <= 10 * U * ref[ok]).all()
    for v in (87.5, 95.0, 103.0, 150.0, 300.0, 3e38, float("inf")):
        z = torch.tensor([[0.0, -v]], device="cuda")
        p = np_(m.mxg_balance_loss_fwd(z, ids, 1.0, status)[2])
        assert p[0] == 1.0 and p[1] == 0.0
    assert int(status.item()) == 0


@pytest.mark.parametrize("T,E", [(40000, 33), (65536, 256), (1000, 5), (19456, 256)])
def test_sums_are_short_chains(T, E):
    """The sums' error goes by the additions that they really take: a lane's tokens (152 blocks of 32 warps of 32 / LPT
    tokens, two a trip), 5 by halves, 32 warps, then 5 blocks in a row and 32 of those."""
    m = require_gpu()
    z, ids = _case(T, E, 2, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, _, sums, _ = m.mxg_balance_loss_fwd(_dev(z), _dev(ids), 0.01, status)
    ref = training.balance_loss(z, ids, 0.01)[2]
    lpt = 1
    while 8 * lpt < E:
        lpt *= 2
    tokens = 152 * 32 * (32 // lpt)
    chain = 2 * -(-T // (2 * tokens)) + 5 + 32 + 5 + 32
    spread = float((z.max(axis=1, keepdims=True) - z).max())
    # a probability: its argument's rounding, 4 U of the exponential, a sum of 8 and up to 5 halvings, reciprocal, product
    p_rel = spread + 4 + 13 + 2 + 1
    assert int(status.item()) == 0
    assert (np.abs(np_(sums) - ref) <= (p_rel + chain) * U * ref).all()
