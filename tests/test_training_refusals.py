"""Refusals of the training operators' entries (no GPU needed): bad arguments
are turned down on the host before anything is launched."""
import ctypes

import pytest
import torch

F = 0x10000             # 32-byte aligned, never dereferenced: the calls fail validation first
BAD = 0x10008
ARG, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


@pytest.fixture(scope="module")
def L():
    from mxfp8_grouped_gemm_gb300 import build
    build.build()
    import mxfp8_grouped_gemm_gb300 as m
    return m.lib()


def test_balance_fwd(L):
    ws = L.mxg_balance_loss_workspace_bytes(64, 8)
    assert ws > 0

    def call(logits=F, ids=F, mask=None, T=64, E=8, k=2, loss=F, counts=F, sums=F, n=F, w=F, wb=ws, st=F):
        return L.mxg_balance_loss_fwd(logits, ids, mask, T, E, k, 0.01, loss, counts, sums, n, w, wb, st, None)

    for name in ("logits", "ids", "loss", "counts", "sums", "n", "w", "st"):
        assert call(**{name: None}) == ARG, name
    for kw in ({"T": 0}, {"T": -1}, {"E": 0}, {"k": 0}):
        assert call(**kw) == ARG
    for kw in ({"E": 257}, {"k": 9}, {"E": 64, "k": 33}, {"T": 1 << 30, "k": 2}):
        assert call(**kw) == SHAPE
    for name in ("logits", "ids", "counts", "sums", "w"):
        assert call(**{name: BAD}) == ALIGN, name
    assert call(wb=ws - 1) == WORKSPACE
    assert L.mxg_balance_loss_workspace_bytes(0, 8) == 0 and L.mxg_balance_loss_workspace_bytes(8, 257) == 0


def test_balance_bwd(L):
    def call(logits=F, mask=None, counts=F, n=F, T=64, E=8, k=2, dloss=None, ids=None, probs=None, dprobs=None, out=F,
             st=F):
        return L.mxg_balance_loss_bwd(logits, mask, counts, n, T, E, k, 0.01, dloss, ids, probs, dprobs, out, st, None)

    for name in ("logits", "counts", "n", "out", "st"):
        assert call(**{name: None}) == ARG, name
    for kw in ({"ids": F}, {"probs": F}, {"dprobs": F}, {"ids": F, "probs": F}, {"probs": F, "dprobs": F}):
        assert call(**kw) == ARG, kw                      # the route's gradient needs all three
    for kw in ({"E": 300}, {"k": 9}):
        assert call(**kw) == SHAPE
    assert call(T=0) == ARG
    for name in ("logits", "counts", "out"):
        assert call(**{name: BAD}) == ALIGN, name
    assert call(ids=BAD, probs=F, dprobs=F) == ALIGN


def test_router_linear_bwd(L):
    ws = L.mxg_router_linear_bwd_workspace_bytes(64, 256, 8)

    def call(x=F, w=F, g=F, dxi=None, T=64, H=256, E=8, dx=F, dw=F, wk=F, wb=ws, st=F):
        return L.mxg_router_linear_bwd(x, w, g, dxi, T, H, E, dx, dw, wk, wb, st, None)

    for name in ("x", "w", "g", "dx", "dw", "wk", "st"):
        assert call(**{name: None}) == ARG, name
    for kw in ({"T": 0}, {"H": 0}, {"E": -3}):
        assert call(**kw) == ARG
    for kw in ({"H": 192}, {"E": 257}):
        assert call(**kw) == SHAPE
    for name in ("x", "w", "g", "dxi", "dx", "dw", "wk"):
        assert call(**{name: BAD}) == ALIGN, name
    assert call(wb=ws - 1) == WORKSPACE
    assert L.mxg_router_linear_bwd_workspace_bytes(0, 256, 8) == 0


def test_muon(L):
    import mxfp8_grouped_gemm_gb300 as m
    ws = L.mxg_muon_workspace_bytes(2, 64, 128)
    assert ws > 0
    good = dict(batch=2, rows=64, cols=128, grad_f32=0, grad=F, mu=0.95, nesterov=1, steps=5, a=1.0, b=0.0, c=0.0,
                scale=1.0, update=F, workspace=F, workspace_bytes=ws, dev_status=F)

    def call(**kw):
        return L.mxg_muon_update(ctypes.byref(m.MuonArgs(**{**good, **kw})), None)

    assert L.mxg_muon_update(None, None) == ARG
    for kw in ({"grad": None}, {"workspace": None}, {"dev_status": None}, {"update": None}, {"momentum_in": F},
               {"w_in": F}, {"w_out": F}, {"steps": 0}, {"steps": 65}, {"rows": 0}, {"batch": -1}):
        assert call(**kw) == ARG, kw
    for kw in ({"batch": 65536}, {"cols": (1 << 21) + 1}, {"batch": 65535, "rows": 1 << 20}):
        assert call(**kw) == SHAPE, kw
    for kw in ({"grad": BAD}, {"momentum_out": BAD}, {"update": BAD}, {"workspace": BAD}, {"w_in": F, "w_out": BAD}):
        assert call(**kw) == ALIGN, kw
    assert call(workspace_bytes=ws - 1) == WORKSPACE
    assert L.mxg_muon_workspace_bytes(0, 4, 4) == 0


def test_python_refuses_wrong_tensors():
    import mxfp8_grouped_gemm_gb300 as m
    z, ids, st = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        m.mxg_balance_loss_fwd(z, ids, 0.01, st)
    with pytest.raises(ValueError, match="shape"):
        m.mxg_balance_loss_fwd(z, ids[:3], 0.01, st)
    with pytest.raises(ValueError, match="shape"):
        m.mxg_balance_loss_bwd(z, torch.zeros(7, dtype=torch.int32), st, 2, 0.01, st)
    x, w = torch.zeros(4, 128).bfloat16(), torch.zeros(8, 128).bfloat16()
    with pytest.raises(ValueError, match="shape"):
        m.mxg_router_linear_bwd(x, w, torch.zeros(4, 7), None, st)
    with pytest.raises(ValueError, match="grad"):
        m.mxg_muon_update(torch.zeros(4), st)
    with pytest.raises(ValueError, match="float32"):
        m.mxg_muon_update(torch.zeros(4, 4).half(), st)
    with pytest.raises(ValueError, match="weights"):
        m.mxg_muon_update(torch.zeros(4, 4), st, weights_out=torch.zeros(4, 4).bfloat16())
    with pytest.raises(ValueError, match="shape"):
        m.mxg_muon_update(torch.zeros(4, 4), st, momentum=torch.zeros(4, 5))
