"""The activations of the products' epilogues in fp32 outputs, densely over their range, against 64 bits."""
import pytest
import torch

import linear_ref as ref
from test_gpu_linear import rnd

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("std", [0.05, 2.0])
def test_activations_in_fp32(bsq, activation, std):
    """The products are the rows' own values (an identity weight) plus a bias: one fp32 number each, which the call
    without an activation gives. GELU's 1 - Phi, which v is multiplied by, is off by at most
      0.75e-7   of the formula (1.5e-7 for erfc)
      4.1e-7    of t, the reciprocal: 2^-23 and two roundings of 2^-24, times 1.72 = the largest t P'(t) / 2
      2.8e-7    of the polynomial's five steps and coefficients: 2^-24 of at most 0.73 each
      1.4e-7    of exp2 (2^-22, of a half) and its argument
      0.9e-7    of the products and the sum behind it: 1e-6 in all.
    The logistic forms have fewer terms: exp2's 2^-22, its argument's roundings times s (1 - s) |x| < 0.23, the
    reciprocal's 2^-23 and two roundings of 2^-24."""
    k = 128
    eye = bsq.quantize("mxfp8", torch.eye(k, device="cuda").to(BF16))
    qx = bsq.quantize("mxfp8", rnd(1, 20000, k, std=std).to(BF16))
    bias = rnd(2, k, std=0.75 * std).to(BF16)
    v = bsq.gemm_act(qx, eye, bias, out_dtype=F32).out.double()
    out = bsq.gemm_act(qx, eye, bias, activation, out_dtype=F32).out
    ref.close(out, ref.act(activation, v), 1e-6 * v.abs() + 1e-37, activation)
    assert bsq.device_status() == 0
