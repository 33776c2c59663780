"""Residual norm with MXFP8 output and its backward on the GPU against the
fp64 oracle, within bounds on the fp32 arithmetic."""
import numpy as np
import pytest
import torch

from gpu_helpers import np_, require_gpu
from oracle import block

pytestmark = pytest.mark.gpu

U = 2.0 ** -24            # half a step of fp32, relative
B = 2.0 ** -8             # of bf16
EPS = 1e-5
CASES = [                 # T, H, residual, fp32 weight
    (1, 8, None, True),
    (1, 4096, "bf16", False),
    (3, 64, "f32", True),
    (17, 72, "bf16", True),           # one past eight lanes
    (33, 128, None, False),
    (100, 136, "f32", False),
    (7, 256, "bf16", False),
    (129, 264, None, True),
    (50, 512, "f32", True),
    (41, 520, "bf16", True),
    (130, 1000, "f32", False),
    (9, 1024, "bf16", False),
    (21, 1032, "bf16", True),         # one past a warp's row
    (700, 2048, "bf16", False),
    (5, 5472, "f32", True),
    (3, 8192, "bf16", True),
    (2, 16376, "f32", False),
    (7, 8200, "bf16", False),         # one past two chunks a thread
    (3, 12288, "bf16", True),
    (2, 12296, "bf16", True),         # one past three
    (200, 9000, None, False),
    (5, 8200, "f32", True),
    (2, 16384, "bf16", True),
    (5003, 128, "bf16", True),        # many rows to a lane group
    (1300, 4096, "bf16", False),
]


def _inputs(T, H, residual, w32, seed=0):
    g = torch.Generator().manual_seed(1000 * H + T + seed)
    loud = 1.0 + 30.0 * (torch.rand(H, generator=g) < 0.02)
    x = torch.randn((T, H), generator=g).bfloat16()
    res = None if residual is None else torch.randn((T, H), generator=g) * loud
    if residual == "bf16":
        res = res.bfloat16()
    w = 1.0 + 0.2 * torch.randn(H, generator=g)
    if T > 2:
        x[1] = 0.0                                         # a row of padding
        if res is not None:
            res[1] = 0.0
    return x, res, (w if w32 else w.bfloat16()), g


def _cuda(t):
    return None if t is None else t.cuda()


def _f64(t):
    return None if t is None else t.double().numpy()


# sum of H squares: a chain of at most 32 in a thread, 5 + 5 halvings, the squares' and r's own roundings (3); times
# 1 / H (2), plus eps (1); under the root half of it, then root and quotient (2)
RSTD = ((32 + 10 + 3 + 3) / 2 + 2) * U


@pytest.mark.parametrize("T,H,residual,w32", CASES)
def test_norm_fwd(T, H, residual, w32):
    m = require_gpu()
    x, res, w, _ = _inputs(T, H, residual, w32)
    codes = H % 128 == 0
    out = m.mxg_rms_norm_fwd(x.cuda(), w.cuda(), EPS, residual=_cuda(res), codes=codes)
    torch.cuda.synchronize()
    r, rstd, y = block.rms_norm(_f64(x), _f64(w), EPS, _f64(res))
    assert (np.abs(np_(out["rstd"]) - rstd) <= RSTD * rstd).all()
    assert (np.abs(np_(out["y"]) - y) <= (B + RSTD + 4 * U) * np.abs(y)).all()
    if res is not None:
        assert out["residual"].dtype == res.dtype
        assert (np.abs(np_(out["residual"]) - r) <= (U if residual == "f32" else B + 2 * U) * np.abs(r)).all()
    if codes:
        for layout in (m.MXG_LAYOUT_CANONICAL,) + ((m.MXG_LAYOUT_MMA,) if T % 128 == 0 else ()):
            other = m.mxg_rms_norm_fwd(x.cuda(), w.cuda(), EPS, residual=_cuda(res), codes=True, bf16=False,
                                       layout=layout)
            assert "y" not in other
            for i in range(0, T, 32):                      # the quantiser takes blocks of 32 rows
                n = min(32, T - i)
                if layout == m.MXG_LAYOUT_CANONICAL:
                    rows = torch.zeros((32, H), dtype=torch.bfloat16, device="cuda")
                    rows[:n] = out["y"][i:i + n]
                    ref = m.mxg_mxfp8_quantize(rows)
                    assert torch.equal(other["q"][i:i + n], ref["q_row"][:n])
                    assert torch.equal(other["s"].view(T, H // 32)[i:i + n], ref["s_row"].view(32, H // 32)[:n])
            if layout == m.MXG_LAYOUT_MMA:
                ref = m.mxg_mxfp8_quantize(out["y"], layout=layout)
                assert torch.equal(other["q"], ref["q_row"]) and torch.equal(other["s"].view(-1), ref["s_row"])
            else:
                assert torch.equal(other["q"], out["q"]) and torch.equal(other["s"], out["s"])


@pytest.mark.parametrize("T,H", [(128, 128), (384, 1024), (256, 4096)])
def test_norm_codes_in_the_mma_layout(T, H):
    m = require_gpu()
    x, res, w, _ = _inputs(T, H, "bf16", False)
    x[3], res[3] = 0.0, 0.0
    x[5] *= 1e4
    out = m.mxg_rms_norm_fwd(x.cuda(), w.cuda() * 300.0, EPS, residual=res.cuda(), codes=True, layout=m.MXG_LAYOUT_MMA)
    ref = m.mxg_mxfp8_quantize(out["y"], layout=m.MXG_LAYOUT_MMA)
    assert torch.equal(out["q"], ref["q_row"]) and torch.equal(out["s"].view(-1), ref["s_row"])


@pytest.mark.parametrize("T,H,residual,w32", CASES)
def test_norm_bwd(T, H, residual, w32):
    m = require_gpu()
    x, res, w, g = _inputs(T, H, residual, w32)
    r = x if res is None else (x.float() + res.float()).to(res.dtype)
    dy = (torch.randn((T, H), generator=g) * 0.01).bfloat16()
    dres = None if residual is None else (torch.randn((T, H), generator=g) * 0.01).to(r.dtype)
    rstd = torch.from_numpy(block.rms_norm(_f64(r), _f64(w), EPS)[1].astype(np.float32))
    dx, dr, dw = m.mxg_rms_norm_bwd(dy.cuda(), r.cuda(), w.cuda(), rstd.cuda(), dresidual=_cuda(dres))
    again = m.mxg_rms_norm_bwd(dy.cuda(), r.cuda(), w.cuda(), rstd.cuda(), dresidual=_cuda(dres))
    torch.cuda.synchronize()
    assert torch.equal(dw, again[2]) and torch.equal(dx, again[0])
    d, dwr = block.rms_norm_grad(_f64(dy), _f64(r), _f64(w), rstd.double().numpy(), _f64(dres))
    xh = np.abs(_f64(r) * rstd.double().numpy()[:, None])
    gw = np.abs(_f64(dy) * _f64(w))
    k = rstd.double().numpy()[:, None]
    mean = np.abs(gw * xh).mean(axis=1, keepdims=True)
    # the mean: terms of 3 roundings, a chain of 32 and 10 halvings, times 1 / H (2); then four operations on the way
    err = k * (3 * U * gw + xh * mean * (3 + 32 + 10 + 2 + 4) * U) + U * np.abs(d)
    assert (np.abs(np_(dx) - d) <= err + B * np.abs(d) + 1e-38).all()
    if residual == "f32":
        assert (np.abs(np_(dr) - d) <= err + 1e-38).all()
    else:
        assert dr is None
    # dweight: a CTA's rows in a chain, up to 16 lane groups, then the CTAs' partials by eight threads and those in order
    ws = m.mxg_rms_norm_bwd_workspace_bytes(T, H)
    ctas = ws // (4 * H)
    chain = -(-T // ctas) + 16 + -(-ctas // 8) + 8 + 3
    assert (np.abs(np_(dw) - dwr) <= chain * U * np.abs(_f64(dy) * xh).sum(axis=0) + 1e-38).all()


def test_norm_in_place():
    m = require_gpu()
    x, res, w, g = _inputs(65, 2048, "bf16", False)
    ref = m.mxg_rms_norm_fwd(x.cuda(), w.cuda(), EPS, residual=res.cuda())
    xc, rc = x.cuda(), res.cuda()
    out = m.mxg_rms_norm_fwd(xc, w.cuda(), EPS, residual=rc, residual_out=rc, y=xc)
    assert out["y"] is xc and torch.equal(xc, ref["y"]) and torch.equal(rc, ref["residual"])
    for dtype in (torch.bfloat16, torch.float32):
        r = ref["residual"].to(dtype)
        dy = torch.randn((65, 2048), generator=g).bfloat16().cuda()
        dres = torch.randn((65, 2048), generator=g).cuda().to(dtype)
        dx, dr, dw = m.mxg_rms_norm_bwd(dy, r, w.cuda(), ref["rstd"], dresidual=dres)
        for into in ("dy", "dresidual"):
            a, b = dy.clone(), dres.clone()
            if dtype == torch.float32:
                got = m.mxg_rms_norm_bwd(a, r, w.cuda(), ref["rstd"], dresidual=b, dx=a, dresidual_out=b)
                assert torch.equal(got[1], dr)
            else:
                got = m.mxg_rms_norm_bwd(a, r, w.cuda(), ref["rstd"], dresidual=b, dx=a if into == "dy" else b)
            assert torch.equal(got[0], dx) and torch.equal(got[2], dw)


@pytest.mark.parametrize("H", [128, 1024, 4096])
def test_norm_bad_rows_stay_their_own(H):
    """NaN and infinity change their own row; rows behind the last are left as they were."""
    m = require_gpu()
    T = 37
    x, res, w, _ = _inputs(T, H, "f32", True)
    good = m.mxg_rms_norm_fwd(x.cuda(), w.cuda(), EPS, residual=res.cuda(), codes=True)
    x[4, 5], x[9, 7] = float("nan"), float("inf")
    big = {n: torch.full((T + 8, H), 77, dtype=t, device="cuda") for n, t in
           (("y", torch.bfloat16), ("q", torch.uint8), ("residual_out", torch.float32))}
    s = torch.full((T + 8, H // 32), 77, dtype=torch.uint8, device="cuda")
    out = m.mxg_rms_norm_fwd(x.cuda(), w.cuda(), EPS, residual=res.cuda(), s=s[:T], **{n: t[:T] for n, t in big.items()})
    keep = [i for i in range(T) if i not in (4, 9)]
    assert torch.equal(out["y"][keep], good["y"][keep]) and torch.equal(out["q"][keep], good["q"][keep])
    assert torch.equal(out["s"][keep], good["s"][keep])
    assert bool(out["y"][4].isnan().all()) and bool(out["y"][9, 7].isnan())
    assert not out["y"][9, :7].any()                      # rstd is zero
    for t in (*big.values(), s):
        assert bool((t[T:] == 77).all())


def test_norm_gradient_is_the_difference():
    """The GPU gradient against central differences of the fp64 norm."""
    m = require_gpu()
    T, H = 3, 40
    x, res, w, g = _inputs(T, H, "f32", True, seed=3)
    r = x.float() + res
    dy, dres = torch.randn((T, H), generator=g).bfloat16(), torch.randn((T, H), generator=g)
    rstd = block.rms_norm(_f64(r), _f64(w), EPS)[1]
    _, d, dw = m.mxg_rms_norm_bwd(dy.cuda(), r.cuda(), w.cuda(), torch.from_numpy(rstd.astype(np.float32)).cuda(),
                                  dresidual=dres.cuda())

    def loss(rr, ww):
        return (block.rms_norm(rr, ww, EPS)[2] * _f64(dy)).sum() + (rr * _f64(dres)).sum()

    h = 1e-6
    R, W = _f64(r), _f64(w)
    for i, j in ((0, 0), (1, 7), (2, 39)):
        e = np.zeros_like(R)
        e[i, j] = h
        diff = (loss(R + e, W) - loss(R - e, W)) / (2 * h)
        assert abs(diff - float(d[i, j])) <= 1e-5 * max(1.0, abs(diff))
        e = np.zeros_like(W)
        e[j] = h
        diff = (loss(R, W + e) - loss(R, W - e)) / (2 * h)
        assert abs(diff - float(dw[j])) <= 1e-5 * max(1.0, abs(diff))


# Widths of every form of the backward (lanes and chunks of a row), with as many rows as make each slot of each CTA's ring
# carry three rows, and the last rows fewer than a CTA takes: rows at a time x CTAs x (2 slots + 1) + a few.
RING = [(136203, 56), (68101, 128), (34051, 248), (21895, 504), (10949, 1000), (5473, 2040), (1369, 8192), (1065, 12280),
        (761, 16384)]


def _ring_inputs(T, H, f32):
    g = torch.Generator(device="cuda").manual_seed(T)
    dt = torch.float32 if f32 else torch.bfloat16
    r, dres = (torch.randn((T, H), generator=g, device="cuda") * s for s in (2.0, 0.01))
    r[T // 2] = 0.0
    dy = (torch.randn((T, H), generator=g, device="cuda") * 0.01).bfloat16()
    w = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")
    r = r.to(dt)
    rstd = (1.0 / (r.double().square().mean(dim=1) + EPS).sqrt()).float()
    return dy, r, w if f32 else w.bfloat16(), rstd, dres.to(dt)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H", RING)
def test_norm_bwd_many_rows_to_a_slot(T, H, f32):
    m = require_gpu()
    dy, r, w, rstd, dres = _ring_inputs(T, H, f32)
    for d_in in (dres, None):
        dx, dr, dw = m.mxg_rms_norm_bwd(dy, r, w, rstd, dresidual=d_in)
        k = rstd.double()[:, None]
        xh, g = r.double() * k, dy.double() * w.double()
        mean = (g * xh).mean(dim=1, keepdim=True)
        d = k * (g - xh * mean)
        if d_in is not None:
            d = d + d_in.double()
        # the roundings of test_norm_bwd
        err = k * (3 * U * g.abs() + xh.abs() * (g * xh).abs().mean(dim=1, keepdim=True) * (3 + 32 + 10 + 2 + 4) * U)
        err += U * d.abs()
        assert bool(((dx.double() - d).abs() <= err + B * d.abs() + 1e-38).all())
        if f32:
            assert bool(((dr.double() - d).abs() <= err + 1e-38).all())
        # dweight: a lane group's rows in a chain, up to 16 groups, the CTAs' partials by 32 threads, and those in 5 halvings
        ctas = m.mxg_rms_norm_bwd_workspace_bytes(T, H) // (4 * H)
        rows = 16 if H <= 64 else 8 if H <= 128 else 4 if H <= 1024 else 1
        chain = -(-T // (ctas * rows)) + rows + -(-ctas // 32) + 5 + 3
        terms = dy.double() * xh
        assert bool(((dw.double() - terms.sum(dim=0)).abs() <= chain * U * terms.abs().sum(dim=0) + 1e-38).all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H", RING)
def test_norm_bwd_in_place_with_rows_on_their_way(T, H, f32):
    """Outputs over dy or dresidual while later rows of both are being copied."""
    m = require_gpu()
    dy, r, w, rstd, dres = _ring_inputs(T, H, f32)
    dx, dr, dw = m.mxg_rms_norm_bwd(dy, r, w, rstd, dresidual=dres)
    for into in ("dy", "dresidual"):
        a, b = dy.clone(), dres.clone()
        if f32:
            got = m.mxg_rms_norm_bwd(a, r, w, rstd, dresidual=b, dx=a if into == "dy" else None, dresidual_out=b)
            assert torch.equal(got[1], dr)
        else:
            got = m.mxg_rms_norm_bwd(a, r, w, rstd, dresidual=b, dx=a if into == "dy" else b)
        assert torch.equal(got[0], dx) and torch.equal(got[2], dw)


@pytest.mark.parametrize("T,H,residual", [(128, 128, "bf16"), (256, 1024, "f32"), (128, 16384, None)])
def test_norm_codes_without_y_in_the_mma_layout(T, H, residual):
    m = require_gpu()
    x, res, w, _ = _inputs(T, H, residual, False)
    out = m.mxg_rms_norm_fwd(x.cuda(), w.cuda(), EPS, residual=_cuda(res))
    only = m.mxg_rms_norm_fwd(x.cuda(), w.cuda(), EPS, residual=_cuda(res), codes=True, bf16=False,
                              layout=m.MXG_LAYOUT_MMA)
    ref = m.mxg_mxfp8_quantize(out["y"], layout=m.MXG_LAYOUT_MMA)
    assert "y" not in only
    assert torch.equal(only["q"], ref["q_row"]) and torch.equal(only["s"].view(-1), ref["s_row"])


@pytest.mark.parametrize("layout", ["canonical", "mma"])
def test_norm_codes_beside_nan(layout):
    """Blocks of y that are NaN in part (weights that are NaN, a row with infinities, whose rstd is zero): the quantiser
    takes the scale from the rest of the block, and so do the codes."""
    m = require_gpu()
    T, H = 128, 256
    x, res, w, _ = _inputs(T, H, "bf16", True)
    w[8:16] = float("nan")
    w[33:64:2] = float("nan")
    w[70] = float("nan")
    w[96:128] = float("nan")
    x[3, 160:168] = float("inf")
    x[4, 192:200:2] = float("-inf")
    layout = m.MXG_LAYOUT_MMA if layout == "mma" else m.MXG_LAYOUT_CANONICAL
    for weight in (w, torch.nan_to_num(w, nan=float("inf")), torch.ones(H)):
        out = m.mxg_rms_norm_fwd(x.cuda(), weight.cuda(), EPS, residual=res.cuda(), codes=True, layout=layout)
        ref = m.mxg_mxfp8_quantize(out["y"], layout=layout)
        assert torch.equal(out["q"], ref["q_row"]) and torch.equal(out["s"].view(-1), ref["s_row"].view(-1))
