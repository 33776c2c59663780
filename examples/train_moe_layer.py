"""One MoE layer trained with everything the library has for it: the router with its balance loss, the grouped MXFP8
expert MLP forward and backward, the dense router backward, and the orthogonalised momentum update of the experts'
and the router's weights.

The task is synthetic: the layer learns a fixed random map of its inputs.  Run on a GB300:

    python examples/train_moe_layer.py [steps]
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


class MoETraining:
    """The layer's weights, momenta and buffers, and one training step over them."""

    def __init__(self, T, H, I, E, k, coef=0.05, lr=0.02, weight_decay=0.01, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std):
            return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()

        self.layer = mxg.GroupedMLP(T, H, I, E, k)
        self.k, self.coef, self.lr, self.weight_decay = k, coef, lr, weight_decay
        self.w_router = weight(E, H, std=H ** -0.5)
        self.w_gate_up = weight(E, 2 * I, H, std=H ** -0.5)
        self.w_down = weight(E, H, I, std=I ** -0.5)
        self.momenta = [torch.zeros(w.shape, device="cuda") for w in (self.w_router, self.w_gate_up, self.w_down)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def update(self, weight, grad, momentum):
        """weight <- weight (1 - lr wd) - lr 0.2 sqrt(longest side) orthogonal(momentum), in place."""
        mxg.mxg_muon_update(grad, self.status, momentum=momentum, scale=0.2 * math.sqrt(max(weight.shape[-2:])),
                            weights=weight, lr=self.lr, weight_decay=self.weight_decay)

    def step(self, x, target, token_mask=None):
        """One step on x, target bf16 [T, H] -> (mean squared error, balance loss, tokens per expert), on the device.
        Tokens that token_mask drops (padding) count in neither loss."""
        layer, k = self.layer, self.k
        logits, ids, probs = mxg.mxg_router_fwd(x, self.w_router, k)
        balance, counts, _, n = mxg.mxg_balance_loss_fwd(logits, ids, self.coef, self.status, token_mask=token_mask)
        y, _ = layer.forward(x, ids, probs, self.w_gate_up, self.w_down)
        err = y.float() - target.float()
        if token_mask is None:
            mse, dy = err.square().mean(), err * (2.0 / err.numel())
        else:
            err = err.masked_fill(token_mask[:, None] == 0, 0.0)
            per = 1.0 / (n.clamp(min=1) * err.shape[1])
            mse, dy = err.square().sum() * per[0], err * (2.0 * per)
        dx, dw_gate_up, dw_down, dprobs = layer.backward(dy.bfloat16())
        # the route's gradient and the balance loss's, on all logits; then through the router's linear layer
        dlogits = mxg.mxg_balance_loss_bwd(logits, counts, n, k, self.coef, self.status, token_mask=token_mask,
                                           route=(ids, probs, dprobs))
        dx, dw_router = mxg.mxg_router_linear_bwd(x, self.w_router, dlogits, dx, self.status, dx=dx)
        self.update(self.w_router, dw_router, self.momenta[0])
        self.update(self.w_gate_up, dw_gate_up, self.momenta[1])
        self.update(self.w_down, dw_down, self.momenta[2])
        return mse, balance, counts


def train(steps=60, T=1024, H=256, I=256, E=8, k=2, seed=0, **kw):
    """-> per step: mean squared error, balance loss, largest share of the routed tokens on one expert."""
    model = MoETraining(T, H, I, E, k, seed=seed, **kw)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher = torch.randn((H, H), generator=gen, device="cuda") * H ** -0.5
    history = []
    for _ in range(steps):
        x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
        target = torch.tanh(x.float() @ teacher).bfloat16()
        mse, balance, counts = model.step(x, target)
        history.append(torch.stack([mse, balance[0], counts.max() / (T * k)]))
    history = torch.stack(history).cpu()
    for status in (int(model.status.item()), model.layer.status()):
        if status != 0:
            raise RuntimeError(mxg.status_string(status))
    return history


if __name__ == "__main__":
    out = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i, (mse, balance, share) in enumerate(out.tolist()):
        if i % 10 == 0 or i + 1 == len(out):
            print(f"step {i:4d}  mse {mse:.4f}  balance loss {balance:.4f}  largest expert share {share:.3f}")
