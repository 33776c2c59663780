"""Balance loss: padding tokens whose route is not valid."""
import numpy as np
import pytest
import torch

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _case(T, E, k, seed):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((T, E)) * 2.0).astype(np.float32)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    c = np.take_along_axis(z.astype(np.float64), ids, axis=1)
    e = np.exp(c - c.max(axis=1, keepdims=True))
    q = (e / e.sum(axis=1, keepdims=True)).astype(np.float32)
    dq = (rng.standard_normal((T, k)) * 0.01 / T).astype(np.float32)
    return z, ids, q, dq, rng.random(T) < 0.8


@pytest.mark.parametrize("T,E,k", [(50, 6, 2), (300, 17, 4), (129, 64, 8), (40, 256, 32)])
def test_padding_tokens_without_a_route(T, E, k):
    """Ids out of range on tokens that the mask drops are padding: neither pass counts, uses or reports them, whatever
    lies in their probs and dprobs."""
    m = require_gpu()
    z, ids, q, dq, mask = _case(T, E, k, E)
    mask[[0, T - 1]] = False
    drop = ~mask
    bad, qn, dqn = ids.copy(), q.copy(), dq.copy()
    bad[drop] = np.where(np.arange(drop.sum())[:, None] % 2 == 0, -1, E + 7)
    qn[drop], dqn[drop] = np.nan, np.inf
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zd, md = _dev(z), _dev(mask)
    loss, counts, _, n = m.mxg_balance_loss_fwd(zd, _dev(bad), 0.5, status, token_mask=md)
    clean_loss, clean_counts, _, _ = m.mxg_balance_loss_fwd(zd, _dev(ids), 0.5, status, token_mask=md)
    assert torch.equal(loss, clean_loss) and torch.equal(counts, clean_counts)
    clean = m.mxg_balance_loss_bwd(zd, counts, n, k, 0.5, status, token_mask=md, route=(_dev(ids), _dev(q), _dev(dq)))
    got = m.mxg_balance_loss_bwd(zd, counts, n, k, 0.5, status, token_mask=md, route=(_dev(bad), _dev(qn), _dev(dqn)))
    assert int(status.item()) == 0
    assert torch.equal(got[md], clean[md]) and not got[~md].any()
    # the same ids on a token that counts are reported
    keep = int(np.flatnonzero(mask)[0])
    bad[keep, 0] = E
    m.mxg_balance_loss_bwd(zd, counts, n, k, 0.5, status, token_mask=md, route=(_dev(bad), _dev(qn), _dev(dqn)))
    assert int(status.item()) == 16
