"""Orthogonalised momentum update: every form that sizes choose between, wide and tall, with the form itself asserted, so
that no change of the rules leaves one untested: the error against the number format's own, both outputs, matrices that
are zero or not finite, gradients of any size, graphs."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import training
from test_gpu_muon import CO, _grad, _orth

pytestmark = pytest.mark.gpu

# batch, short, long; CTAs of a matrix on the chip, columns of a tile, whether a contraction of X X^T is shared
FORMS = {
    "chip1 two parts": (3, 48, 64, 1, 0, False),
    "chip2 two parts": (3, 64, 96, 2, 0, False),
    "chip8 two parts": (40, 48, 4096, 8, 0, False),
    "chip16 two parts": (3, 48, 8192, 16, 0, False),
    "chip1": (3, 128, 256, 1, 0, False),
    "chip2": (60, 112, 1008, 2, 0, False),
    "chip4": (30, 112, 2000, 4, 0, False),
    "chip8": (3, 128, 2048, 8, 0, False),
    "chip16": (3, 112, 8192, 16, 0, False),
    "one tile two parts": (200, 48, 8208, 0, 128, False),
    "one tile two parts shared": (3, 48, 8208, 0, 128, True),
    "one tile two parts shared odd": (3, 47, 9001, 0, 128, True),
    "one tile two parts odd": (160, 31, 8211, 0, 128, False),
    "one tile": (170, 96, 1008, 0, 128, False),
    "one tile odd": (161, 127, 1001, 0, 128, False),
    "one tile shared": (3, 112, 9008, 0, 128, True),
    "tiles of 64": (3, 208, 304, 0, 64, False),
    "tiles of 64 odd": (3, 201, 303, 0, 64, False),
    "tiles of 64 shared": (3, 208, 3008, 0, 64, True),
    "tiles of 128": (20, 304, 304, 0, 128, False),
    "tiles of 128 odd": (20, 303, 305, 0, 128, False),
    "tiles of 128, blocks": (24, 528, 1040, 0, 128, False),
    "tiles of 128 shared": (3, 608, 2000, 0, 128, True),
    "pairs": (24, 512, 1024, 0, 256, False),
    "pairs, blocks": (12, 768, 1536, 0, 256, False),
    "pairs ragged": (30, 400, 1600, 0, 256, False),
    "pairs odd": (30, 401, 1601, 0, 256, False),
    "pairs shared": (8, 400, 4000, 0, 256, True),
    "pairs shared odd": (8, 399, 4001, 0, 256, True),
}
ALL = pytest.mark.parametrize("name", FORMS)
WIDE_TALL = pytest.mark.parametrize("tall", [False, True])
# what bf16 rounding alone leaves of a matrix's norm: sqrt(1/12) of a unit in the last place, on average
ROUNDING = 1.67e-3


def _case(m, name, tall):
    batch, short, long_, cluster, tile, shared = FORMS[name]
    rows, cols = (long_, short) if tall else (short, long_)
    form = m.mxg_muon_form(batch, rows, cols)
    assert (form["cluster"], form["tile"], form["shares"] > 1) == (cluster, tile, shared), form
    assert form["parts"] == (2 if short <= 64 else 1)
    return batch, rows, cols


def _format(u):
    """The error that the number format alone makes on each matrix, relative to its norm."""
    short, long_ = sorted(u.shape[1:])
    x_parts = 2 if short <= 64 else 1
    b_parts = 2 if short <= 64 or (short < 120 and long_ > 512) else 1
    ref = [training.orthogonalise(a, 5, CO) for a in u]
    return [np.linalg.norm(training.orthogonalise_in_fp16(a, 5, CO, x_parts, b_parts) - r) / np.linalg.norm(r)
            for a, r in zip(u, ref)]


def _as_the_format(got, u, margin=1.05):
    """The roundings are the simulated ones but where a sum in fp32 lands on the other side of a tie, and the sums' own
    errors are far below them: 5 % of margin."""
    for g, a, e in zip(np_(got).astype(np.float64), u, _format(u)):
        r = training.orthogonalise(a, 5, CO)
        assert np.linalg.norm(g - r) <= margin * e * np.linalg.norm(r), (np.linalg.norm(g - r) / np.linalg.norm(r), e)


@ALL
@WIDE_TALL
def test_error_is_the_formats(name, tall):
    m = require_gpu()
    batch, rows, cols = _case(m, name, tall)
    g = torch.from_numpy(_grad(batch, rows, cols, 11)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    upd = m.mxg_muon_update(g, status)
    ends = [0, batch - 1]
    _as_the_format(upd[ends], g[ends].double().cpu().numpy())
    assert torch.equal(upd, m.mxg_muon_update(g, status)) and int(status.item()) == 0


@WIDE_TALL
@pytest.mark.parametrize("batch,short,long_,cluster,shares,most", [
    (3, 48, 64, 1, False, 0.025),
    (3, 64, 96, 2, False, 0.025),
    (3, 48, 1024, 8, False, 0.025),
    (3, 48, 4500, 16, False, 0.025),
    (17, 56, 4608, 0, True, 0.025),
    (160, 40, 4200, 0, False, 0.1),
])
def test_two_parts_leave_the_results_rounding(batch, short, long_, cluster, shares, most, tall):
    """Short sides up to 64: every product of parts is there.  The update is the exact one's rounding but for elements
    next to a tie.  A sum of n columns in one accumulator is cut by 1.5e-8 n / 16, at most 30 times that in X: 2e-5 at
    768 columns, where 1 to 2 % of the elements fall otherwise, and 1e-4 (5 %) at 4200.  A lost product moves 12 % and
    more, one of X X^T 5 to 15 % up to 1024 columns and 2 to 3 % above 4000 (simulated)."""
    m = require_gpu()
    rows, cols = (long_, short) if tall else (short, long_)
    form = m.mxg_muon_form(batch, rows, cols)
    assert form["parts"] == 2 and form["cluster"] == cluster and (form["shares"] > 1) == shares
    g = torch.from_numpy(_grad(batch, rows, cols, 19)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    upd = np_(m.mxg_muon_update(g, status)[[0, batch - 1]])
    exact = training.bf16_round(_orth(g[[0, batch - 1]].double().cpu().numpy()))
    assert (upd != exact).mean() <= most and int(status.item()) == 0


@ALL
@WIDE_TALL
def test_weights_alone_in_place_and_beside_the_update(name, tall):
    """The last product's epilogue for weights: to another matrix, in place, and with the update beside it (which takes
    another path out): the same bits, and the oracle's weights."""
    m = require_gpu()
    batch, rows, cols = _case(m, name, tall)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(batch, rows, cols, 12)).cuda()
    scale, lr, wd = 0.2 * np.sqrt(max(rows, cols)), 0.05, 0.3
    w = (torch.from_numpy(_grad(batch, rows, cols, 13)) * 10).bfloat16().cuda()
    kw = dict(scale=scale, lr=lr, weight_decay=wd)
    out = m.mxg_muon_update(g, status, weights=w, weights_out=torch.empty_like(w), **kw)
    upd, both = torch.empty_like(w), torch.empty_like(w)
    m.mxg_muon_update(g, status, weights=w, weights_out=both, update=upd, **kw)
    alone = m.mxg_muon_update(g, status, scale=scale)
    here = w.clone()
    assert m.mxg_muon_update(g, status, weights=here, **kw).data_ptr() == here.data_ptr()
    assert torch.equal(out, here) and torch.equal(out, both) and torch.equal(alone, upd)
    ends = [0, batch - 1]
    W, u = w[ends].double().cpu().numpy(), g[ends].double().cpu().numpy()
    for got, a, b, e in zip(np_(out[ends]).astype(np.float64), W, u, _format(u)):
        step = lr * scale * training.orthogonalise(b, 5, CO)
        ref = a * (1 - lr * wd) - step
        # the step has the format's error (its own bf16 rounding included), the weights their rounding
        bound = 1.05 * np.hypot(ROUNDING * np.linalg.norm(ref), e * np.linalg.norm(step))
        assert np.linalg.norm(got - ref) <= bound
        assert np.linalg.norm(step) > 0.1 * np.linalg.norm(ref)          # it shows
    assert int(status.item()) == 0


@ALL
@WIDE_TALL
def test_zero_and_bad_matrices_stay_alone(name, tall):
    m = require_gpu()
    batch, rows, cols = _case(m, name, tall)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(batch, rows, cols, 14)).cuda()
    g[1] = 0.0
    clean = m.mxg_muon_update(g, status)
    for bad in (float("nan"), float("inf")):
        g[2, rows - 1, cols // 3] = bad
        upd = m.mxg_muon_update(g, status)
        keep = [i for i in range(batch) if i != 2]
        assert not upd[1].any() and torch.equal(clean[keep], upd[keep]) and torch.isnan(upd[2]).any()
    assert int(status.item()) == 0


@ALL
@WIDE_TALL
@pytest.mark.parametrize("scale", [1e-42, 1e-25, 1e30])
def test_any_size_of_gradient(name, tall, scale):
    m = require_gpu()
    batch, rows, cols = _case(m, name, tall)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(batch, rows, cols, 15)).double() * 1e6
    g = (g * scale).float().cuda()
    upd = m.mxg_muon_update(g, status)
    _as_the_format(upd[:1], g[:1].cpu().double().numpy())
    assert int(status.item()) == 0


@ALL
@WIDE_TALL
def test_captured_in_a_graph(name, tall):
    m = require_gpu()
    batch, rows, cols = _case(m, name, tall)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(_grad(batch, rows, cols, 16)).cuda()
    mom, out = torch.zeros_like(g), torch.empty(g.shape, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(m.mxg_muon_workspace_bytes(batch, rows, cols), dtype=torch.uint8, device="cuda")
    m.mxg_muon_update(g, status, momentum=mom, update=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mxg_muon_update(g, status, momentum=mom, update=out, workspace=ws)
    other = mom.clone()
    for seed in (17, 18):
        g.copy_(torch.from_numpy(_grad(batch, rows, cols, seed)))
        graph.replay()
        expected = m.mxg_muon_update(g, status, momentum=other)
        assert torch.equal(out, expected) and torch.equal(mom, other)
    assert int(status.item()) == 0


@WIDE_TALL
@pytest.mark.parametrize("batch,short,long_", [(2, 512, 1024), (1, 128, 256), (1, 100, 3000), (24, 512, 1024)])
@pytest.mark.parametrize("rank", [1, 8, 64])
def test_low_rank_gradients_have_the_formats_error(batch, short, long_, rank, tall):
    """A gradient of few tokens: X0's rounding fills the empty directions, and five steps multiply what is in them by
    3.4445^5 = 485.  With short sides over 64 that is up to 15 % of the update for rank 1, and no more than the number
    format's roundings give."""
    m = require_gpu()
    rng = np.random.default_rng(rank)
    rows, cols = (long_, short) if tall else (short, long_)
    u = rng.standard_normal((batch, rows, rank)) @ rng.standard_normal((batch, rank, cols))
    g = torch.from_numpy((u * 1e-3).astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    upd = m.mxg_muon_update(g, status)
    # the roundings of the first steps are multiplied too, those that fall otherwise among them
    _as_the_format(upd[:1], g[:1].double().cpu().numpy(), 1.1)
    assert int(status.item()) == 0


@WIDE_TALL
@pytest.mark.parametrize("short,long_,rank", [(48, 512, 1), (64, 4096, 4), (40, 8208, 2)])
def test_low_rank_gradients_in_two_parts(short, long_, rank, tall):
    """Short sides up to 64 are held in two parts: the update's own rounding is all that shows."""
    m = require_gpu()
    rng = np.random.default_rng(rank)
    rows, cols = (long_, short) if tall else (short, long_)
    u = rng.standard_normal((1, rows, rank)) @ rng.standard_normal((1, rank, cols))
    g = torch.from_numpy(u.astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _as_the_format(m.mxg_muon_update(g, status), g.double().cpu().numpy())
    assert int(status.item()) == 0
