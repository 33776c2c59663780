"""Orthogonalised momentum update: long sides whose sums take more matrix instructions than one accumulator should."""
import pytest
import torch

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

CO = (3.4445, -4.7750, 2.0315)


def _exact(u):
    x = u.double() / torch.linalg.norm(u.double())
    for _ in range(5):
        a = x @ x.T
        x = CO[0] * x + (CO[1] * a + CO[2] * a @ a) @ x
    return x


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("batch,m,n", [
    (152, 4, 1 << 21),          # as many matrices as SMs: none is idle to share a contraction; the longest side there is
    (152, 100, 32769),          # one tile, one part: three shares, several of them to a CTA
    (1, 100, 1 << 20),          # shared by idle SMs in any case
    (80, 130, 65600),           # several tiles, several shares to a CTA or pair
    (1, 140, 1 << 17),
])
def test_long_side(batch, m, n, tall):
    """The tensor cores cut their running sums (1.5e-8 of the result per instruction): 2e-3 of a diagonal element of
    X X^T over 2^21 columns, which five steps magnify (3.7e-2 of the update).  In accumulators of at most 1024
    instructions (4096 where there are several tiles) less than 6e-4 of the update is left beside its rounding
    (1.66e-3) and, with one part, the operands' (2.4e-3 together)."""
    mx = require_gpu()
    rows, cols = (n, m) if tall else (m, n)
    gen = torch.Generator(device="cuda").manual_seed(m)
    g = torch.randn((batch, rows, cols), generator=gen, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    upd = mx.mxg_muon_update(g, status)
    form = mx.mxg_muon_form(batch, rows, cols)
    assert form["cluster"] == 0 and -(-n // form["shares"]) <= (16384 if m <= 128 else 65536)
    for b in {0, batch - 1}:
        ref = _exact(g[b].T if tall else g[b])
        err = float(((upd[b].T if tall else upd[b]).double() - ref).norm() / ref.norm())
        assert err <= (1.8e-3 if form["parts"] == 2 else 2.6e-3), err
    assert torch.equal(upd, mx.mxg_muon_update(g, status))
    assert int(status.item()) == 0
