"""The operators around the linear layers working together: training steps of the example's block."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("expert_block_step", os.path.join(ROOT, "examples", "expert_block_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_steps_reduce_the_loss():
    import block_scaled_precision_bsq_gb300 as bsq

    ex = _example()
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(700, 256, device="cuda", generator=gen).to(torch.bfloat16)
    target = torch.randn(700, 256, device="cuda", generator=gen).to(torch.bfloat16)
    block = ex.ExpertBlock(width=256, hidden=512, experts=4)
    losses = []
    for _ in range(6):
        loss, norm = block.step(x, target, lr=2.0, max_norm=0.05)
        losses.append(float(loss))
        clipped = float(torch.linalg.vector_norm(torch.cat([g.reshape(-1).double() for g in block.grads.values()])))
        assert clipped <= 0.05 * (1 + 1e-5) and float(norm) >= clipped * (1 - 1e-5)
        assert all(torch.isfinite(g).all() for g in block.grads.values()) and torch.isfinite(block.dx.float()).all()
    assert bsq.device_status() == 0
    # every step follows the gradient a short way: the loss falls each time
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_gradient_of_the_norms_and_gate_against_autograd():
    """The same step in fp32 torch, for the parameters that no quantized layer stands behind."""
    ex = _example()
    import block_scaled_precision_bsq_gb300 as bsq

    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(300, 256, device="cuda", generator=gen)
    h = torch.randn(300, 256, device="cuda", generator=gen)
    target = torch.randn(300, 256, device="cuda", generator=gen)
    p = {k: (v + 0.1 * torch.randn(v.shape, device="cuda", generator=gen)).requires_grad_()
         for k, v in ex.ExpertBlock(width=256, hidden=512, experts=4).params.items() if v.dim() == 1}
    ln = torch.nn.functional.layer_norm
    n = ln(h, (256,), p["post_weight"], p["post_bias"], 1e-6)
    y = ln(x + p["gate"] * n, (256,), p["out_weight"], p["out_bias"], 1e-6)
    ((y - target).square().sum() / 2).backward()
    kw = {k: v.detach() for k, v in dict(post_weight=p["post_weight"], post_bias=p["post_bias"], gate=p["gate"],
                                         pre_weight=p["out_weight"], pre_bias=p["out_bias"]).items()}
    f = bsq.block_norm(h, x, post_norm=True, **kw)
    r = bsq.block_norm_backward(None, f.y - target, f.x_out, h, f.stats, post_norm=True, **kw)
    # fp32 on both sides, sums of 300 terms: 1e-4 of the largest value is far above either's error
    for got, name in ((r.dpost_weight, "post_weight"), (r.dpost_bias, "post_bias"), (r.dgate, "gate"),
                      (r.dpre_weight, "out_weight"), (r.dpre_bias, "out_bias")):
        want = p[name].grad
        assert (got - want).abs().max() <= 1e-4 * want.abs().max(), name
