"""Dense router backward: gradients that are not finite."""
import numpy as np
import pytest
import torch

import synthetic
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [5, 8, 100])
def test_every_nan_stays_a_nan(E):
    """A NaN may have set bits in any place of its significand: cut into bf16 parts it is a NaN still, in its token's
    dx and its expert's dW and nowhere else; an infinity gives nothing finite there."""
    m = require_gpu()
    T, H = 200, 256
    x, w = synthetic.random_bf16((T, H), 1).cuda(), synthetic.random_bf16((E, H), 2, std=0.02).cuda()
    rng = np.random.default_rng(3)
    clean = (rng.standard_normal((T, E)) * 1e-3).astype(np.float32)
    bad = clean.copy()
    bits = bad.view(np.uint32)
    nans = {(3, 0): 0x7F800001, (70, 1): 0xFF80FFFF, (71, 2): 0x7FC00000, (199, 3): 0x7F801000}
    for (t, e), b in nans.items():
        bits[t, e] = b
    bad[100, 4] = np.inf
    assert np.isnan(bad).sum() == len(nans)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx0, dw0 = m.mxg_router_linear_bwd(x, w, torch.from_numpy(clean).cuda(), None, status)
    dx, dw = m.mxg_router_linear_bwd(x, w, torch.from_numpy(bad).cuda(), None, status)
    torch.cuda.synchronize()
    for t, e in nans:
        assert torch.isnan(dx[t]).all() and torch.isnan(dw[e]).all(), hex(nans[t, e])
    assert not torch.isfinite(dx[100]).any() and not torch.isfinite(dw[4]).any()
    rows = [t for t in range(T) if t not in (3, 70, 71, 100, 199)]
    assert torch.equal(dx[rows], dx0[rows]) and torch.equal(dw[5:], dw0[5:])
    assert int(status.item()) == 0
