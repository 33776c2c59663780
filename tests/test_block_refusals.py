"""Refusals of the block operators' entries (no GPU needed): bad arguments are
turned down on the host before anything is launched."""
import ctypes

import pytest
import torch

F = 0x10000             # 32-byte aligned, never dereferenced: the calls fail validation first
BAD = 0x10008
ARG, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


@pytest.fixture(scope="module")
def m():
    from mxfp8_grouped_gemm_gb300 import build
    build.build()
    import mxfp8_grouped_gemm_gb300 as m
    return m


def test_route_fwd(m):
    def call(logits=F, bias=None, T=64, E=16, k=2, score=0, groups=1, top=1, gt=1, renorm=1, scale=1.0, ids=F, probs=F):
        a = m.RouteScoresFwdArgs(T, E, k, score, groups, top, gt, renorm, scale, logits, bias, ids, probs)
        return m.lib().mxg_route_scores_fwd(ctypes.byref(a), None)

    assert m.lib().mxg_route_scores_fwd(None, None) == ARG
    for name in ("logits", "ids", "probs"):
        assert call(**{name: None}) == ARG and call(**{name: BAD}) == ALIGN, name
    assert call(bias=BAD) == ALIGN
    for kw in ({"T": 0}, {"T": -1}, {"E": 0}, {"k": 0}, {"score": 2}, {"score": -1}, {"scale": 0.0}, {"scale": -1.0},
               {"scale": float("nan")}, {"scale": float("inf")}, {"groups": 0}, {"top": 0}, {"gt": 0}, {"gt": 3}):
        assert call(**kw) == ARG, kw
    for kw in ({"E": 257}, {"k": 17}, {"E": 64, "k": 33}, {"groups": 3}, {"groups": 32}, {"groups": 4, "top": 5},
               {"groups": 8, "top": 1, "k": 3}, {"groups": 16, "top": 4, "gt": 2}):
        assert call(**kw) == SHAPE, kw


def test_route_bwd(m):
    def call(logits=F, ids=F, probs=F, dprobs=F, add=None, T=64, E=16, k=2, score=1, renorm=1, scale=1.0, out=F, st=F):
        a = m.RouteScoresBwdArgs(T, E, k, score, renorm, scale, logits, ids, probs, dprobs, add, out, st)
        return m.lib().mxg_route_scores_bwd(ctypes.byref(a), None)

    assert m.lib().mxg_route_scores_bwd(None, None) == ARG
    for name in ("logits", "ids", "probs", "dprobs", "out", "st"):
        assert call(**{name: None}) == ARG, name
    for name in ("logits", "ids", "probs", "dprobs", "add", "out"):
        assert call(**{name: BAD}) == ALIGN, name
    for kw in ({"T": 0}, {"k": 0}, {"score": 5}, {"scale": 0.0}):
        assert call(**kw) == ARG, kw
    for kw in ({"E": 300}, {"k": 17}):
        assert call(**kw) == SHAPE, kw


def test_norm_fwd(m):
    def call(**kw):
        a = m.RmsNormFwdArgs(**(dict(T=64, H=256, x=F, weight=F, eps=1e-6, y=F) | kw))
        return m.lib().mxg_rms_norm_fwd(ctypes.byref(a), None)

    assert m.lib().mxg_rms_norm_fwd(None, None) == ARG
    for kw in ({"x": None}, {"weight": None}, {"y": None}, {"q": F}, {"s": F}, {"residual_out": F}, {"T": 0}, {"H": 0},
               {"H": -8}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"q": F, "s": F, "layout": 2}):
        assert call(**kw) == ARG, kw
    for kw in ({"H": 255}, {"H": 16392}, {"H": 64, "q": F, "s": F}, {"T": 65, "q": F, "s": F, "layout": 1}):
        assert call(**kw) == SHAPE, kw
    for kw in ({"x": BAD}, {"weight": BAD}, {"y": BAD}, {"residual": BAD}, {"residual": F, "residual_out": BAD},
               {"q": BAD, "s": F}, {"q": F, "s": BAD}, {"rstd": BAD}):
        assert call(**kw) == ALIGN, kw


def test_norm_bwd(m):
    L = m.lib()
    ws = L.mxg_rms_norm_bwd_workspace_bytes(64, 256)
    assert ws > 0

    def call(**kw):
        a = m.RmsNormBwdArgs(**(dict(T=64, H=256, dy=F, r=F, weight=F, rstd=F, dx=F, dweight=F, workspace=F,
                                     workspace_bytes=ws) | kw))
        return L.mxg_rms_norm_bwd(ctypes.byref(a), None)

    assert L.mxg_rms_norm_bwd(None, None) == ARG
    for name in ("dy", "r", "weight", "rstd", "dx", "dweight", "workspace"):
        assert call(**{name: None}) == ARG and call(**{name: BAD}) == ALIGN, name
    for kw in ({"T": 0}, {"H": 0}, {"dresidual_out": F}):
        assert call(**kw) == ARG, kw
    for kw in ({"H": 100}, {"H": 20000}):
        assert call(**kw) == SHAPE, kw
    assert call(dresidual=BAD) == ALIGN and call(r_f32=1, dresidual_out=BAD) == ALIGN
    assert call(workspace_bytes=ws - 1) == WORKSPACE
    for T, H in ((0, 256), (64, 0), (64, 12), (64, 16392)):
        assert L.mxg_rms_norm_bwd_workspace_bytes(T, H) == 0


def test_clip(m):
    L = m.lib()
    ws = L.mxg_grad_norm_workspace_bytes(2)
    assert ws > 0 and L.mxg_grad_norm_workspace_bytes(0) == 0 == L.mxg_grad_norm_workspace_bytes(-1)

    def refs(**kw):
        t = (m.TensorRef * 2)()
        for r in t:
            r.ptr, r.out, r.numel, r.f32 = F, F, 100, 1
        for name, v in kw.items():
            setattr(t[1], name, v)
        return t

    def norm(t=None, n=2, to=F, w=F, wb=ws, **kw):
        return L.mxg_grad_norm(refs(**kw) if t is None else t, n, to, w, wb, None)

    def clip(n=2, most=1.0, by=None, to=F, w=F, wb=ws, **kw):
        return L.mxg_grad_clip(refs(**kw), n, most, by, to, w, wb, None)

    for call in (norm, clip):
        for kw in ({"n": 0}, {"n": -1}, {"numel": -1}, {"f32": 2}, {"ptr": None}, {"w": None}):
            assert call(**kw) == ARG, kw
        for kw in ({"ptr": F + 2}, {"ptr": F + 1, "f32": 0}, {"w": BAD}, {"to": BAD}):
            assert call(**kw) == ALIGN, kw
        assert call(numel=1 << 50) == SHAPE
        assert call(wb=ws - 1) == WORKSPACE
    assert L.mxg_grad_norm(None, 2, F, F, ws, None) == ARG and norm(to=None) == ARG
    for kw in ({"most": 0.0}, {"most": -1.0}, {"most": float("nan")}, {"out": None}, {"by": F, "to": F}):
        assert clip(**kw) == ARG, kw
    assert clip(out=F + 2) == ALIGN and clip(by=BAD, to=None) == ALIGN


def test_binding(m):
    z, i, p = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    st = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: m.mxg_route_scores_fwd(z, 2), lambda: m.mxg_route_scores_bwd(z, i, p, p, st),
                 lambda: m.mxg_rms_norm_fwd(z.bfloat16(), torch.ones(8)), lambda: m.mxg_grad_norm([z]),
                 lambda: m.mxg_rms_norm_bwd(z.bfloat16(), z.bfloat16(), torch.ones(8), torch.ones(4)),
                 lambda: m.mxg_grad_clip([z], 1.0)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    x = z.bfloat16()
    for call, text in ((lambda: m.mxg_route_scores_fwd(z, 2, score="tanh"), "softmax"),
                       (lambda: m.mxg_route_scores_fwd(z[0], 2), "two dimensions"),
                       (lambda: m.mxg_route_scores_fwd(z, 2, bias=torch.zeros(7)), "bias"),
                       (lambda: m.mxg_route_scores_fwd(z, 3, ids=i), "ids"),
                       (lambda: m.mxg_route_scores_bwd(z, i, p[:2], p, st), "probs"),
                       (lambda: m.mxg_route_scores_bwd(z, i, p, p, st, dlogits_in=z[:2]), "dlogits_in"),
                       (lambda: m.mxg_rms_norm_fwd(x, torch.ones(7)), "weight"),
                       (lambda: m.mxg_rms_norm_fwd(x, torch.ones(8).half()), "weight"),
                       (lambda: m.mxg_rms_norm_fwd(x, torch.ones(8), residual_out=z), "residual_out"),
                       (lambda: m.mxg_rms_norm_fwd(x, torch.ones(8), q=i), "together"),
                       (lambda: m.mxg_rms_norm_fwd(x, torch.ones(8), y=x, bf16=False), "bf16"),
                       (lambda: m.mxg_rms_norm_bwd(x, x, torch.ones(8), torch.ones(4), dresidual_out=z), "fp32"),
                       (lambda: m.mxg_rms_norm_bwd(x, x, torch.ones(8), torch.ones(3)), "rstd"),
                       (lambda: m.mxg_grad_norm([]), "no gradients"), (lambda: m.mxg_grad_norm([z.half()]), "float16"),
                       (lambda: m.mxg_grad_clip([z], 1.0, out=[]), "outputs"),
                       (lambda: m.mxg_grad_clip([z], 1.0, norm=p, norm_out=p), "norm_out")):
        with pytest.raises(ValueError, match=text):
            call()


def test_clip_workspace_of_any_count(m):
    """Eight bytes for each of 608 blocks, per 512 tensors: also where n + 511 passes 31 bits."""
    for n in (1, 512, 513, 10 ** 6, 2 ** 31 - 512, 2 ** 31 - 511, 2 ** 31 - 1):
        assert m.mxg_grad_norm_workspace_bytes(n) == -(-n // 512) * 608 * 8, n
