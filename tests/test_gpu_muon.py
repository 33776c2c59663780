"""Orthogonalised momentum update on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import training

pytestmark = pytest.mark.gpu

CO = (3.4445, -4.7750, 2.0315)
U = 2.0 ** -24
CASES = [                       # batch, rows, cols
    (1, 1, 1),
    (1, 1, 300),                # one row
    (2, 300, 1),                # one column
    (1, 8, 4096),               # a router's weight
    (3, 15, 17),
    (4, 128, 256),              # tiny layer's W_down
    (4, 512, 128),              # tiny layer's W_gate_up, taller than wide
    (2, 129, 255),              # one past a tile, one short of two
    (2, 333, 1001),
    (1, 1001, 333),
    (70, 64, 96),               # many small matrices
    (1, 1024, 2816),            # several tiles of the wide kernel
    (80, 260, 520),             # the CTA-pair kernel on ragged tiles
]
# fp16 operands: X, A and B are each rounded to 11 bits (2e-4 rms) once per step and the polynomial's
# derivative is at most ~5 on A and ~3.4 on X, so a step adds about 1e-3; five of them and the bf16 output
# (1.7e-3) stay below 1e-2 of the result's norm.  Single elements: eight standard deviations of that.
REL = 1e-2


def _grad(batch, rows, cols, seed, strong=2.0):
    rng = np.random.default_rng(seed)
    r = max(1, min(rows, cols) // 16)
    u = rng.standard_normal((batch, rows, r)) @ (rng.standard_normal((batch, r, cols)) * (strong / np.sqrt(r)))
    return ((u + rng.standard_normal((batch, rows, cols))) * 1e-3).astype(np.float32)


def _close(got, ref, name=""):
    got, rms = np_(got).astype(np.float64), np.sqrt(np.mean(ref * ref))
    assert np.linalg.norm(got - ref) <= REL * np.linalg.norm(ref), (name, np.linalg.norm(got - ref) / np.linalg.norm(ref))
    assert (np.abs(got - ref) <= 8 * REL * rms + 2.0 ** -8 * np.abs(ref)).all(), name


def _orth(u, scale=1.0, steps=5):
    return np.stack([training.orthogonalise(a, steps, CO) for a in u]) * scale


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("batch,rows,cols", CASES)
def test_update(batch, rows, cols, f32):
    m = require_gpu()
    g = torch.from_numpy(_grad(batch, rows, cols, rows + cols))
    g = (g if f32 else g.bfloat16()).cuda()
    mom = torch.from_numpy(_grad(batch, rows, cols, 7 + rows) * 5).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mom_out = torch.empty_like(mom)
    upd = m.mxg_muon_update(g, status, momentum=mom, momentum_out=mom_out, scale=0.7)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    G, M = g.double().cpu().numpy(), mom.double().cpu().numpy()
    new, u = training.momentum(G, M, 0.95, True)
    assert (np.abs(np_(mom_out) - new) <= 3 * U * (np.abs(G) + 0.95 * np.abs(M))).all()
    _close(upd, _orth(u, 0.7))


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("rows,cols", [(96, 160), (160, 96)])
def test_momentum_forms_and_weights(rows, cols, nesterov):
    """No momentum yet, momentum in place, the weights updated in the same call."""
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(2, rows, cols, 3)).cuda()
    G = g.double().cpu().numpy()
    _close(m.mxg_muon_update(g, status), _orth(G), "no momentum")
    mom = torch.empty_like(g)
    upd = m.mxg_muon_update(g, status, momentum_out=mom, nesterov=nesterov)
    assert torch.equal(mom, g)                                        # mom' = g
    _close(upd, _orth(G), "first step")
    w = (torch.from_numpy(_grad(2, rows, cols, 4)) * 20).bfloat16().cuda()
    W = w.double().cpu().numpy()
    M = mom.double().cpu().numpy()
    out = m.mxg_muon_update(g * 0.5, status, momentum=mom, mu=0.9, nesterov=nesterov, weights=w, lr=0.1,
                            weight_decay=0.2, scale=0.5)
    torch.cuda.synchronize()
    assert out.data_ptr() == w.data_ptr() and int(status.item()) == 0
    new, u = training.momentum(0.5 * G, M, 0.9, nesterov)
    assert (np.abs(np_(mom) - new) <= 3 * U * (np.abs(G) + np.abs(M))).all()
    step = _orth(u, 0.05)
    ref = W * (1 - 0.1 * 0.2) - step
    assert (np.abs(np_(w) - ref) <= 2.0 ** -8 * np.abs(ref) + 8 * REL * np.sqrt(np.mean(step ** 2))).all()


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_steps(steps):
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(2, 100, 300, 5)).cuda()
    _close(m.mxg_muon_update(g, status, steps=steps), _orth(g.double().cpu().numpy(), 1.0, steps))


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-15, 1e12, 1e25, 1e34])
def test_gradients_of_any_size(scale):
    """The norm neither overflows nor underflows: the update does not depend on the gradient's size."""
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = np.random.default_rng(2).standard_normal((1, 40, 90)).astype(np.float32) * np.float32(1e3)
    gs = (g.astype(np.float64) * scale).astype(np.float32)            # 1e-42: whole multiples of the smallest subnormal
    upd = m.mxg_muon_update(torch.from_numpy(gs).cuda(), status)
    torch.cuda.synchronize()
    _close(upd, _orth(gs.astype(np.float64)))


def test_idle_expert_and_bad_expert_stay_alone():
    """A zero matrix gives zeros; NaN or infinity in one matrix leaves the others bit-identical."""
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = _grad(5, 130, 200, 6)
    g[1] = 0.0
    clean = m.mxg_muon_update(torch.from_numpy(g).cuda(), status)
    g[3, 17, 5] = np.nan
    g[4, 0, 0] = np.inf
    upd = m.mxg_muon_update(torch.from_numpy(g).cuda(), status)
    torch.cuda.synchronize()
    assert not clean[1].any() and not upd[1].any()
    assert torch.equal(clean[[0, 1, 2]], upd[[0, 1, 2]])
    assert torch.isnan(upd[3]).any() and torch.isnan(upd[4]).any()
    assert int(status.item()) == 0


def test_singular_values_go_to_one():
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    upd = m.mxg_muon_update(torch.from_numpy(_grad(1, 200, 700, 8)).cuda(), status)
    s = np.linalg.svd(np_(upd)[0].astype(np.float64), compute_uv=False)
    # the polynomial's fixed band is about 0.68 .. 1.13
    assert s.min() > 0.6 and s.max() < 1.25


def test_repeatable_two_dimensional_and_on_another_stream():
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(1, 300, 500, 9)).cuda()
    a = m.mxg_muon_update(g, status)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = m.mxg_muon_update(g[0], status, stream=s)
    s.synchronize()
    assert b.shape == (300, 500) and torch.equal(a[0], b)


def test_workspace_is_not_exceeded():
    """Canaries behind the workspace and the outputs."""
    m = require_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for batch, rows, cols in [(2, 129, 255), (3, 37, 41), (80, 260, 520)]:
        n = batch * rows * cols
        ws_bytes = m.mxg_muon_workspace_bytes(batch, rows, cols)
        ws = torch.full((ws_bytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        buf = torch.full((n + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
        mom = torch.full((n + 1024,), 3.0, device="cuda")
        g = torch.from_numpy(_grad(batch, rows, cols, 1)).cuda()
        m.mxg_muon_update(g, status, momentum_out=mom[:n].view(batch, rows, cols),
                          update=buf[:n].view(batch, rows, cols), workspace=ws[:ws_bytes])
        torch.cuda.synchronize()
        assert (ws[ws_bytes:] == 0x5A).all() and (buf[n:] == 7.0).all() and (mom[n:] == 3.0).all()
