"""The block operators together, as a model uses them: the training block against the fp64 oracle, the inference path
on MXFP8 rows bit for bit, graphs, streams and threads."""
import os
import sys
import threading

import numpy as np
import pytest
import torch

import synthetic
from conftest import ROOT
from gpu_helpers import np_, require_gpu
from oracle import block, moe

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))


def _rms(a, r):
    return float(np.sqrt(np.mean((a - r) ** 2)) / np.sqrt(np.mean(r ** 2)))


def test_training_block_against_the_oracle():
    """Forward and every gradient of the block, the experts' MXFP8 arithmetic taken by the oracle as well."""
    require_gpu()
    import train_moe_block
    T, H, I, E, k = 256, 128, 256, 8, 2
    b = train_moe_block.MoEBlock(T, H, I, E, k, groups=4, top_groups=2, scale=1.5, seed=5)
    gen = torch.Generator().manual_seed(6)
    b.bias.copy_(torch.randn(E, generator=gen) * 0.1)
    b.norm.copy_(1.0 + 0.1 * torch.randn(H, generator=gen))
    x, residual, dout, dres = (torch.randn((T, H), generator=gen).bfloat16() for _ in range(4))
    out, stream = b.forward(x.cuda(), residual.cuda())
    dx, grads = b.backward(dout.cuda(), dres.cuda())
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0 and b.layer.status() == 0

    w = {n: t.double().cpu().numpy() for n, t in (("norm", b.norm), ("router", b.w_router), ("gu", b.w_gate_up),
                                                   ("down", b.w_down), ("bias", b.bias))}
    r, _, _ = block.rms_norm(x.double().numpy(), w["norm"], b.eps, residual.double().numpy())
    n, logits, ids, probs, _ = b.saved
    y = n["y"].double().cpu().numpy()
    # the route is the oracle's on the GPU's logits, which are within the router's own bound of the oracle's
    z = np_(logits).astype(np.float64)
    assert _rms(z, y @ w["router"].T) < 1e-5
    ids_ref, probs_ref = block.route(z, k, "sigmoid", w["bias"], 4, 2, 2, True, 1.5)
    assert np.array_equal(np_(ids), ids_ref)
    ctx = moe.mlp_fwd(y, ids_ref.astype(np.int32), probs_ref, w["gu"], w["down"])
    g = moe.mlp_bwd(ctx, dout.double().numpy())
    assert _rms(np_(out), ctx["y"]) <= 2e-2 and _rms(np_(stream), r) <= 2.0 ** -8
    dlogits = block.route_grad(z, ids_ref, probs_ref, g["dprobs"], "sigmoid", True, 1.5)
    dy = g["dx"] + dlogits @ w["router"]
    dr, dnorm = block.rms_norm_grad(dy, n["residual"].double().cpu().numpy(), w["norm"],
                                    n["rstd"].double().cpu().numpy(), dres.double().numpy())
    for name, got, ref in (("dx", dx, dr), ("norm", grads[0], dnorm), ("router", grads[1], dlogits.T @ y),
                           ("gate_up", grads[2], g["dw_gate_up"]), ("down", grads[3], g["dw_down"])):
        assert _rms(np_(got).astype(np.float64), ref) <= 2e-2, name

    before = [t.clone() for t in grads]
    ref = block.grad_norm([t.double().cpu().numpy() for t in before])
    b.max_norm = ref / 2
    norm = b.update(grads)
    assert abs(float(norm) - ref) <= 1e-6 * ref
    for a, c in zip(grads, before):
        assert _rms(np_(a).astype(np.float64), c.double().cpu().numpy() / 2) <= 2.0 ** -8
    load = np_(b.saved[4])
    moved = np_(b.bias) - w["bias"]
    assert np.abs(moved - 0.01 * np.sign(load.mean() - load)).max() < 1e-6


def test_example_runs_and_repeats():
    require_gpu()
    import train_moe_block
    a = train_moe_block.train(steps=12)
    assert torch.isfinite(a).all() and torch.equal(a, train_moe_block.train(steps=12))


def test_inference_on_mxfp8_rows():
    """Norm codes gathered by expert and taken as they are give what the bf16 rows give, bit for bit."""
    m = require_gpu()
    T, H, I, E, k = 300, 256, 256, 8, 2
    x, residual = synthetic.random_bf16((T, H), 1).cuda(), synthetic.random_bf16((T, H), 2).cuda()
    w = (1.0 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(3))).cuda()
    w_router = synthetic.random_bf16((E, H), 4, std=0.05).cuda()
    w_gu = synthetic.random_bf16((E, 2 * I, H), 5, std=0.05).cuda()
    w_d = synthetic.random_bf16((E, H, I), 6, std=0.05).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = m.mxg_rms_norm_fwd(x, w, residual=residual, codes=True)
    logits, _, _ = m.mxg_router_fwd(n["y"], w_router, k)
    ids, probs = m.mxg_route_scores_fwd(logits, k, score="sigmoid", groups=4, top_groups=2, scale=2.0)
    perm = m.mxg_route_permute(ids, E, status)
    experts = m.GroupedExperts(T * k, H, I, E)
    experts.quantize_weights(w_gu, w_d)
    p_rows = m.mxg_gather_rows(probs.view(-1), perm["src_of_row"], status)
    rows = m.mxg_gather_rows(n["y"], perm["src_of_row"], status, div=k)
    a = m.mxg_combine(experts.forward(rows, perm["split_sizes"], p_rows, save_for_backward=False), perm["row_of_src"], k,
                      status)
    q, s = (m.mxg_gather_rows(n[c], perm["src_of_row"], status, div=k) for c in ("q", "s"))
    b = m.mxg_combine(experts.forward_mx(q, s, perm["split_sizes"], p_rows), perm["row_of_src"], k, status)
    only = m.mxg_rms_norm_fwd(x, w, residual=residual, codes=True, bf16=False)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and experts.status() == 0
    assert torch.equal(a, b) and bool(a.any())
    assert torch.equal(only["q"], n["q"]) and torch.equal(only["s"], n["s"])


class _Work:
    """One call of each operator on inputs of its own, and what it gives alone."""

    def __init__(self, m, seed, T=700, H=2048, E=64, k=8):
        self.m, self.k = m, k
        g = torch.Generator().manual_seed(seed)
        self.x, self.res, self.dy = (torch.randn((T, H), generator=g).bfloat16().cuda() for _ in range(3))
        self.w = torch.randn(H, generator=g).cuda()
        self.z, self.bias = torch.randn((T, E), generator=g).cuda(), (torch.randn(E, generator=g) * 0.1).cuda()
        self.dp = torch.randn((T, k), generator=g).cuda()
        self.grads = [torch.randn(s, generator=g).cuda().to(t) for s, t in
                      (((300000,), torch.float32), ((77, 99), torch.bfloat16), ((5,), torch.float32))]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.expected = self.run()
        torch.cuda.synchronize()

    def run(self, **kw):
        m = self.m
        n = m.mxg_rms_norm_fwd(self.x, self.w, residual=self.res, codes=True, **kw)
        back = m.mxg_rms_norm_bwd(self.dy, n["residual"], self.w, n["rstd"], dresidual=self.res, **kw)
        ids, p = m.mxg_route_scores_fwd(self.z, self.k, score="sigmoid", bias=self.bias, groups=8, top_groups=4, **kw)
        d = m.mxg_route_scores_bwd(self.z, ids, p, self.dp, self.status, score="sigmoid", **kw)
        if kw:                                             # a stream of its own: outputs are made on the current one
            out = [torch.zeros_like(t) for t in self.grads]
            torch.cuda.current_stream().synchronize()
        else:
            out = [torch.empty_like(t) for t in self.grads]
        norm, out = m.mxg_grad_clip(self.grads, 3.0, out=out, **kw)
        return [n["y"], n["q"], n["s"], n["residual"], n["rstd"], back[0], back[2], ids, p, d, norm,
                m.mxg_grad_norm(self.grads, **kw), *out]

    def check(self, got):
        assert all(torch.equal(a, b) for a, b in zip(got, self.expected)) and int(self.status.item()) == 0


def test_streams_in_turn():
    m = require_gpu()
    work = [_Work(m, i) for i in range(3)]
    streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], [], []]
    for _ in range(15):
        for s, w, o in zip(streams, work, outs):
            with torch.cuda.stream(s):
                o.append(w.run())
    torch.cuda.synchronize()
    for w, o in zip(work, outs):
        for got in o:
            w.check(got)


def test_given_stream():
    m = require_gpu()
    w, s = _Work(m, 8), torch.cuda.Stream()
    got = w.run(stream=s)
    s.synchronize()
    w.check(got)


def test_threads():
    m = require_gpu()
    work, outs, errors, start = [_Work(m, 10 + i) for i in range(3)], [[], [], []], [], threading.Barrier(3)

    def body(i):
        try:
            start.wait()
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(15):
                    outs[i].append(work[i].run())
                torch.cuda.current_stream().synchronize()
        except BaseException as e:                         # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for w, o in zip(work, outs):
        for got in o:
            w.check(got)


def test_graphs_with_eager_calls_between():
    """Two captured graphs replayed in turn, with calls outside them."""
    m = require_gpu()
    work = [_Work(m, 20), _Work(m, 21), _Work(m, 22)]
    graphs, captured = [], []
    for w in work[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            captured.append(w.run())
        graphs.append(g)
    for _ in range(5):
        for c in captured:
            for t in c:
                t.zero_()
        for g in graphs:
            g.replay()
        work[2].check(work[2].run())
        torch.cuda.synchronize()
        for w, c in zip(work, captured):
            w.check(c)
    # new values in the captured inputs
    fresh = _Work(m, 23)
    with torch.no_grad():
        for name in ("x", "res", "dy", "w", "z", "bias", "dp"):
            getattr(work[0], name).copy_(getattr(fresh, name))
        for a, b in zip(work[0].grads, fresh.grads):
            a.copy_(b)
    graphs[0].replay()
    torch.cuda.synchronize()
    fresh.check(captured[0])


def test_long_offsets():
    """Element numbers that pass 31 bits: 140000 rows of 16384, and logits of 2^31 / 200 tokens by 256."""
    m = require_gpu()
    T, H = 140000, 16384
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    last = torch.randn((3, H), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    x[-3:] = last
    w = torch.ones(H, device="cuda")
    n = m.mxg_rms_norm_fwd(x, w, codes=True)
    ref = m.mxg_rms_norm_fwd(last, w, codes=True)
    for name in ("y", "q", "s", "rstd"):
        assert torch.equal(n[name][-3:], ref[name]), name
    dy = torch.zeros_like(x)
    dy[-3:] = last
    dx, _, dw = m.mxg_rms_norm_bwd(dy, x, w, n["rstd"])
    dx2, _, dw2 = m.mxg_rms_norm_bwd(last, last, w, ref["rstd"])
    assert torch.equal(dx[-3:], dx2) and not dx[:-3].any()
    assert float((dw - dw2).abs().max()) <= 1e-5 * float(dw2.abs().max())
    norm, (got,) = m.mxg_grad_clip([x], 1.0)
    assert abs(float(norm) - float(last.double().square().sum().sqrt())) <= 1e-5 * float(norm)
    assert float((got[-3:].double() - last.double() / float(norm)).abs().max()) <= 2.0 ** -8 * 5 / float(norm)
    del x, dy, n, dx, got
    T, E, k = 10737418, 256, 4
    z = torch.zeros((T, E), device="cuda")
    tail = torch.randn((5, E), generator=torch.Generator().manual_seed(2)).cuda()
    z[-5:] = tail
    ids, p = m.mxg_route_scores_fwd(z, k, score="sigmoid")
    ids2, p2 = m.mxg_route_scores_fwd(tail, k, score="sigmoid")
    assert torch.equal(ids[-5:], ids2) and torch.equal(p[-5:], p2)
    assert torch.equal(ids[:3].cpu(), torch.arange(k, dtype=torch.int32).expand(3, k)) and float(p[0, 0]) == 0.25
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = m.mxg_route_scores_bwd(z, ids, p, p, st, score="sigmoid", dlogits=z)
    assert torch.equal(d[-5:], m.mxg_route_scores_bwd(tail, ids2, p2, p2, st, score="sigmoid")) and int(st.item()) == 0
