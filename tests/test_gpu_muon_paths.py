"""Orthogonalised momentum update: the forms that sizes choose between (matrices that stay on the chip with one to
eight CTAs each; single-tile and tiled products, on one SM or a pair; outputs that TMA cannot address), each wide and
tall, against the fp64 oracle within test_gpu_muon's tolerances."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import training
from test_gpu_muon import REL, U, _close, _grad, _orth

pytestmark = pytest.mark.gpu

CASES = [                       # batch, short, long
    (2, 9, 33),                 # on the chip, one CTA, high and low parts
    (3, 60, 130),               # three boxes of columns over clusters
    (1, 64, 513),               # one column past a CTA's share
    (1, 31, 2050),
    (2, 17, 4096),              # the longest side that stays on the chip
    (200, 33, 70),              # more matrices than SMs
    (1, 65, 90),                # on the chip, one part
    (2, 128, 512),
    (1, 101, 1025),
    (1, 128, 4095),
    (1, 40, 4100),              # one tile of A, its contraction shared by several CTAs, high and low parts
    (3, 100, 5003),             # the same with one part
    (90, 100, 700),             # one tile of A, too many matrices for clusters
    (2, 129, 300),              # two row tiles, of which the second holds one row
    (1, 256, 257),
    (40, 257, 511),             # pairs, three 256-blocks on and above the diagonal
]


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("batch,m,n", CASES)
def test_forms(batch, m, n, tall):
    mx = require_gpu()
    rows, cols = (n, m) if tall else (m, n)
    g = torch.from_numpy(_grad(batch, rows, cols, 3 * m + n)).cuda()
    mom = torch.from_numpy(_grad(batch, rows, cols, 5 * m + n) * 3).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(mom)
    upd = mx.mxg_muon_update(g, status, momentum=mom, momentum_out=out, scale=1.3)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    G, M = g.double().cpu().numpy(), mom.double().cpu().numpy()
    new, u = training.momentum(G, M, 0.95, True)
    assert (np.abs(np_(out) - new) <= 3 * U * (np.abs(G) + 0.95 * np.abs(M))).all()
    _close(upd, _orth(u, 1.3))
    again = mx.mxg_muon_update(g, status, momentum=mom, momentum_out=out, scale=1.3)
    assert torch.equal(upd, again)


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("batch,m,n", [
    (1, 130, 3001),             # tiles of 64 columns, every one's contraction shared; odd rows
    (2, 600, 2000),             # of 128, shared
    (8, 400, 4000),             # of 256 on pairs, shared
    (8, 399, 4001),
    (20, 300, 300),             # of 128, not shared
    (70, 200, 200),             # of 256 on pairs, not shared, one tile each
    (30, 128, 2000),            # on the chip, clusters of four
    (19, 64, 1024),             # the same, where eight would not fit at once
    (38, 100, 1000),            # clusters of two
    (3, 48, 8192),              # clusters of sixteen, high and low parts
    (2, 101, 5001),             # the same with one part, the last CTAs without columns
    (9, 60, 4500),              # too many of them to stay on the chip
    (9, 100, 4500),
    (1, 40, 8200),              # too long for it
    (1, 100, 9001),
])
def test_many_matrices_and_long_ones(batch, m, n, tall):
    """The forms that need many or long matrices; the oracle on the first and the last one."""
    mx = require_gpu()
    rows, cols = (n, m) if tall else (m, n)
    g = torch.from_numpy(_grad(batch, rows, cols, 7 * m + n)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    upd = mx.mxg_muon_update(g, status, scale=0.7)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ends = sorted({0, batch - 1})
    _close(upd[ends], _orth(g[ends].double().cpu().numpy(), 0.7))
    assert torch.equal(upd, mx.mxg_muon_update(g, status, scale=0.7))


@pytest.mark.parametrize("batch,m,n", [(3, 90, 6000), (2, 96, 3000), (1, 80, 9000), (40, 100, 700)])
@pytest.mark.parametrize("tall", [False, True])
def test_few_strong_directions(batch, m, n, tall):
    """Short sides of 65 to 119, where B's rounding would be the largest error: with B in two parts the update's own
    rounding (1.66e-3), A's (1.1e-3 of the result) and X's (0.7e-3) are left, 2.1e-3 together; with a tenth of margin."""
    mx = require_gpu()
    rows, cols = (n, m) if tall else (m, n)
    g = torch.from_numpy(_grad(batch, rows, cols, 9 * m + n)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    upd = mx.mxg_muon_update(g, status)
    ends = sorted({0, batch - 1})
    got, ref = np_(upd[ends]).astype(np.float64), _orth(g[ends].double().cpu().numpy())
    assert int(status.item()) == 0
    assert np.linalg.norm(got - ref) <= 2.3e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("rows,cols", [(48, 96), (96, 48), (100, 5000), (200, 304), (304, 200), (201, 303)])
def test_update_and_weights_together(rows, cols):
    """Both outputs of one call are what each gives alone."""
    import ctypes
    mx = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(2, rows, cols, 21)).cuda()
    w = (torch.from_numpy(_grad(2, rows, cols, 22)) * 20).bfloat16().cuda()
    upd = mx.mxg_muon_update(g, status, scale=0.3)
    w1 = mx.mxg_muon_update(g, status, scale=0.3, weights=w, weights_out=torch.empty_like(w), lr=0.1, weight_decay=0.2)
    both, w2 = torch.empty_like(upd), torch.empty_like(w)
    got = mx.mxg_muon_update(g, status, scale=0.3, update=both, weights=w, weights_out=w2, lr=0.1, weight_decay=0.2)
    torch.cuda.synchronize()
    assert got is w2 and int(status.item()) == 0
    assert torch.equal(both, upd) and torch.equal(w1, w2)
    step = _orth(g.double().cpu().numpy(), 0.03)
    ref = w.double().cpu().numpy() * (1 - 0.1 * 0.2) - step
    assert (np.abs(np_(w2) - ref) <= 2.0 ** -8 * np.abs(ref) + 8 * REL * np.sqrt(np.mean(step ** 2))).all()


@pytest.mark.parametrize("batch,rows,cols", [(3, 30, 200), (3, 700, 90), (3, 100, 4500), (3, 200, 333), (40, 260, 300)])
def test_zero_and_bad_matrices_stay_alone(batch, rows, cols):
    """In every form: zeros give zeros, NaN in one matrix leaves the others bit-identical."""
    mx = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = _grad(batch, rows, cols, 31)
    g[1] = 0.0
    clean = mx.mxg_muon_update(torch.from_numpy(g).cuda(), status)
    g[2, rows // 2, cols // 3] = np.nan
    upd = mx.mxg_muon_update(torch.from_numpy(g).cuda(), status)
    torch.cuda.synchronize()
    keep = [i for i in range(batch) if i != 2]
    assert not upd[1].any() and torch.equal(clean[keep], upd[keep]) and torch.isnan(upd[2]).any()
    assert int(status.item()) == 0


@pytest.mark.parametrize("rows,cols", [(20, 100), (100, 20), (90, 200), (30, 5000), (150, 160)])
@pytest.mark.parametrize("scale", [1e-42, 1e-25, 1e30])
def test_any_size_of_gradient(rows, cols, scale):
    mx = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = np.random.default_rng(rows).standard_normal((1, rows, cols)) * 1e3 * scale
    g = g.astype(np.float32)
    upd = mx.mxg_muon_update(torch.from_numpy(g).cuda(), status)
    torch.cuda.synchronize()
    _close(upd, _orth(g.astype(np.float64)))


def test_captured_in_a_graph():
    """Every form only enqueues work: captured once, replayed on new gradients."""
    mx = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for batch, rows, cols in [(2, 64, 96), (2, 128, 1024), (1, 100, 4500), (2, 333, 1001)]:
        g = torch.from_numpy(_grad(batch, rows, cols, 1)).cuda()
        ws = torch.empty(mx.mxg_muon_workspace_bytes(batch, rows, cols), dtype=torch.uint8, device="cuda")
        out = torch.empty(g.shape, dtype=torch.bfloat16, device="cuda")
        mx.mxg_muon_update(g, status, update=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mx.mxg_muon_update(g, status, update=out, workspace=ws)
        g.copy_(torch.from_numpy(_grad(batch, rows, cols, 2)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.mxg_muon_update(g, status))
