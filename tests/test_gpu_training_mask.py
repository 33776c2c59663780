"""The training example's token mask: padding trains nothing."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_padding_targets_do_not_matter():
    require_gpu()
    import train_moe_layer
    T, H = 512, 256
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    target = torch.tanh(torch.randn((T, H), generator=gen, device="cuda")).bfloat16()
    mask = torch.rand(T, generator=gen, device="cuda") < 0.75
    other = torch.where(mask[:, None], target, torch.full_like(target, float("nan")))
    out = []
    for y in (target, other):
        model = train_moe_layer.MoETraining(T, H, 256, 8, 2)
        losses = [torch.stack([v.reshape(()) for v in model.step(x, y, mask)[:2]]) for _ in range(3)]
        out.append([*losses, model.w_router, model.w_gate_up, model.w_down, *model.momenta])
        assert int(model.status.item()) == 0 and model.layer.status() == 0
    assert all(torch.isfinite(t).all() for t in out[0])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_nothing_but_padding():
    require_gpu()
    import train_moe_layer
    T, H = 256, 256
    x = torch.randn((T, H), device="cuda").bfloat16()
    model = train_moe_layer.MoETraining(T, H, 256, 8, 2, weight_decay=0.0)
    before = [w.clone() for w in (model.w_router, model.w_gate_up, model.w_down)]
    mse, balance, counts = model.step(x, x, torch.zeros(T, dtype=torch.bool, device="cuda"))
    assert float(mse) == 0.0 and float(balance) == 0.0 and not counts.any()
    assert all(torch.equal(a, b) for a, b in zip(before, (model.w_router, model.w_gate_up, model.w_down)))
