"""clip_grad_norm where the coefficient's quotient has no value of its own."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_an_infinite_limit_clips_nothing_whatever_the_norm():
    import block_scaled_precision_bsq_gb300 as bsq

    for bad in (math.inf, -math.inf):
        for kind in (2.0, math.inf):
            g = torch.randn(5000, device="cuda")
            g[77] = bad
            keep, out = g.clone(), torch.empty_like(g)
            assert float(bsq.clip_grad_norm([g], math.inf, kind, outs=[out])) == math.inf
            assert torch.equal(out, keep)
            bsq.clip_grad_norm([g], math.inf, kind)
            assert torch.equal(g, keep)
    g = torch.randn(5000, device="cuda")
    g[5] = math.nan  # a NaN norm makes every gradient NaN, whatever the limit
    bsq.clip_grad_norm([g], math.inf)
    assert g.isnan().all()


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_zero_gradients_stay_zero_under_a_limit_of_zero(eps):
    import block_scaled_precision_bsq_gb300 as bsq

    for dtype in (torch.bfloat16, torch.float32):
        g = torch.zeros(1000, dtype=dtype, device="cuda")
        out = torch.full_like(g, 7.0)
        assert float(bsq.clip_grad_norm([g], 0.0, eps=eps, outs=[out])) == 0.0
        assert (out == 0).all()
        bsq.clip_grad_norm([g], 0.0, eps=eps)
        assert (g == 0).all()


@pytest.mark.parametrize("count", [1, 64, 65, 1100])
def test_a_norm_equal_to_the_limit_changes_nothing(count):
    """norm + eps == max_norm: a coefficient of one, also over several launches."""
    import block_scaled_precision_bsq_gb300 as bsq

    gs = [torch.full((4,), 0.5, device="cuda") for _ in range(count)]
    norm = float(bsq.grad_norm(gs))
    keep = [g.clone() for g in gs]
    bsq.clip_grad_norm(gs, norm, eps=0.0)
    assert all(torch.equal(a, b) for a, b in zip(gs, keep))
    bsq.clip_grad_norm(gs, norm / 2, eps=0.0)
    assert all(torch.equal(a, b / 2) for a, b in zip(gs, keep))
