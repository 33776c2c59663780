"""One MoE block of a model trained: residual stream and norm, the router with sigmoid scores, groups and a bias that
balances the load, the grouped MXFP8 expert MLP forward and backward, the gradients clipped by their norm, and the
orthogonalised momentum update.

    h = residual + x;  y = norm(h);  out = h + experts(y, route(y))

The task is synthetic: the block learns a fixed random map of its inputs.  Run on a GB300:

    python examples/train_moe_block.py [steps]
"""
from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mxfp8_grouped_gemm_gb300 as mxg  # noqa: E402


class MoEBlock:
    """The block's weights, momenta and buffers, its forward and backward, and one training step over them."""

    def __init__(self, T, H, I, E, k, groups=1, top_groups=1, score="sigmoid", scale=1.0, bias_rate=0.01, lr=0.02,
                 max_norm=1.0, eps=1e-6, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std):
            return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()

        self.layer = mxg.GroupedMLP(T, H, I, E, k)
        self.route = dict(score=score, renormalize=True, scale=scale)
        self.groups = dict(groups=groups, top_groups=top_groups, group_top=2 if E // groups > 1 else 1)
        self.eps, self.bias_rate, self.lr, self.max_norm = eps, bias_rate, lr, max_norm
        self.norm = torch.ones(H, device="cuda")
        self.bias = torch.zeros(E, device="cuda")                     # chooses experts, carries no gradient
        self.w_router = weight(E, H, std=H ** -0.5)
        self.w_gate_up = weight(E, 2 * I, H, std=H ** -0.5)
        self.w_down = weight(E, H, I, std=I ** -0.5)
        self.momenta = [torch.zeros(w.shape, device="cuda") for w in (self.w_router, self.w_gate_up, self.w_down)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def forward(self, x, residual):
        """x, residual bf16 [T, H] -> (the experts' output, the residual stream, bf16 [T, H] each)."""
        n = mxg.mxg_rms_norm_fwd(x, self.norm, self.eps, residual=residual)
        logits, _, _ = mxg.mxg_router_fwd(n["y"], self.w_router, self.layer.k)
        ids, probs = self.layer.route_scores(logits, bias=self.bias, **self.route, **self.groups)
        out, split_sizes = self.layer.forward(n["y"], ids, probs, self.w_gate_up, self.w_down)
        self.saved = n, logits, ids, probs, split_sizes
        return out, n["residual"]

    def backward(self, dout, dresidual):
        """Gradients of both outputs -> (gradient of x and of residual alike, those of norm, w_router, w_gate_up, w_down)."""
        n, logits, ids, probs, _ = self.saved
        dy, dw_gate_up, dw_down, dprobs = self.layer.backward(dout)
        dlogits = mxg.mxg_route_scores_bwd(logits, ids, probs, dprobs, self.status, **self.route)
        dy, dw_router = mxg.mxg_router_linear_bwd(n["y"], self.w_router, dlogits, dy, self.status, dx=dy)
        dx, _, dnorm = mxg.mxg_rms_norm_bwd(dy, n["residual"], self.norm, n["rstd"], dresidual=dresidual)
        return dx, [dnorm, dw_router, dw_gate_up, dw_down]

    def update(self, grads):
        """Clips the gradients by their norm (in place) and updates weights and bias -> the norm before clipping."""
        norm, (dnorm, *rest) = mxg.mxg_grad_clip(grads, self.max_norm)
        self.norm -= self.lr * dnorm
        for w, g, m in zip((self.w_router, self.w_gate_up, self.w_down), rest, self.momenta):
            mxg.mxg_muon_update(g, self.status, momentum=m, scale=0.2 * math.sqrt(max(w.shape[-2:])), weights=w, lr=self.lr)
        # an expert with fewer tokens than the mean is preferred from now on
        load = self.saved[4].float()
        self.bias += self.bias_rate * torch.sign(load.mean() - load)
        return norm

    def step(self, x, residual, target):
        """One step towards out + residual stream = target -> (mean squared error, gradient norm, tokens per expert)."""
        out, stream = self.forward(x, residual)
        err = out.float() + stream.float() - target.float()
        derr = (err * (2.0 / err.numel())).bfloat16()
        _, grads = self.backward(derr, derr)
        return err.square().mean(), self.update(grads), self.saved[4]


def train(steps=60, T=1024, H=256, I=256, E=16, k=2, seed=0, **kw):
    """-> per step: mean squared error, gradient norm, largest share of the routed tokens on one expert."""
    block = MoEBlock(T, H, I, E, k, seed=seed, **({"groups": 4, "top_groups": 2} | kw))
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher = torch.randn((H, H), generator=gen, device="cuda") * H ** -0.5
    history = []
    for _ in range(steps):
        x, residual = (torch.randn((T, H), generator=gen, device="cuda").bfloat16() for _ in range(2))
        h = x.float() + residual.float()
        mse, norm, load = block.step(x, residual, (h + torch.tanh(h @ teacher)).bfloat16())
        history.append(torch.stack([mse, norm[0], load.max() / (T * k)]))
    history = torch.stack(history).cpu()
    for status in (int(block.status.item()), block.layer.status()):
        if status != 0:
            raise RuntimeError(mxg.status_string(status))
    return history


if __name__ == "__main__":
    out = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i, (mse, norm, share) in enumerate(out.tolist()):
        if i % 10 == 0 or i + 1 == len(out):
            print(f"step {i:4d}  mse {mse:.4f}  gradient norm {norm:.4f}  largest expert share {share:.3f}")
