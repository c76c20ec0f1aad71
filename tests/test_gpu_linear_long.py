"""Products with activation, residual and experts whose buffers pass 2^32 bytes and 2^31 values: kept arguments, residuals
and gradients with a row stride, column sums, weight gradients in fp32."""
import pytest
import torch

import linear_ref as ref
from test_gpu_linear import rnd, segments

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ROWS, N, K = 270_001, 8192, 128


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


def picked():
    return torch.cat([torch.arange(0, 300), torch.arange(262_100, 262_200), torch.arange(ROWS - 300, ROWS)]).cuda()


def strided(seed, cols, dtype=BF16):
    """A matrix of ROWS x cols whose rows are 8 values further apart, made in pieces."""
    wide = torch.empty(ROWS, cols + 8, device="cuda", dtype=dtype)
    for i in range(0, ROWS, 30_000):
        wide[i:i + 30_000] = rnd(seed + i, min(30_000, ROWS - i), cols + 8, std=1.5)
    return wide[:, 8:]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_residual_and_kept_argument_pass_32_bits(bsq, dtype):
    qx, qw = bsq.quantize("mxfp8", rnd(1, ROWS, K).to(BF16)), bsq.quantize("mxfp8", rnd(2, N, K, std=0.1).to(BF16))
    residual = strided(3, N, dtype)
    r = bsq.gemm_act(qx, qw, None, "silu", residual, save_pre=True)
    at, b = picked(), ref.decode(qw)
    a = ref.decode(bsq.QTensor(qx.fmt, ROWS, K, qx.codes, qx.scales))[at]
    v, size = a @ b.t(), a.abs() @ b.abs().t()
    off = ref.SUM * size + 2.0 ** -23 * v.abs()
    ref.close(r.pre[at], v, off + ref.half_step(BF16) * v.abs(), "pre")
    want = ref.act("silu", v) + residual[at].to(F64)
    off = 1.13 * off + ref.ACT * v.abs() + 2.0 ** -23 * want.abs()
    ref.close(r.out[at], want, 1.01 * off + ref.half_step(dtype) * want.abs(), "out")
    assert bsq.device_status() == 0


def test_kept_argument_of_experts_passes_32_bits(bsq):
    c, o, _, spans = segments([5, ROWS - 9, 4])
    qx, qw = bsq.quantize("mxfp8", rnd(1, ROWS, K).to(BF16)), bsq.quantize("mxfp8", rnd(2, 3 * N, K, std=0.1).to(BF16))
    r = bsq.expert_gemm(qx, qw, c, o, None, "relu", save_pre=True)
    at, a, b = picked(), ref.decode(qx), ref.decode(qw)
    for e, (lo, hi) in enumerate(spans):
        i = at[(at >= lo) & (at < hi)]
        w = b[e * N:(e + 1) * N]
        v, size = a[i] @ w.t(), a[i].abs() @ w.abs().t()
        off = ref.SUM * size + ref.half_step(BF16) * v.abs()
        ref.close(r.pre[i], v, off, "pre of expert %d" % e)
        ref.close(r.out[i], v.clamp(min=0), off, "out of expert %d" % e)
    assert bsq.device_status() == 0


def test_gradient_and_column_sums_pass_32_bits(bsq):
    qdy = bsq.quantize("mxfp8", rnd(1, ROWS, K, std=1e-3).to(BF16))
    qw = bsq.quantize("mxfp8", rnd(2, N, K, std=0.1).to(BF16))
    pre = strided(3, N)
    r = bsq.gemm_act_backward(qdy, qw, pre, "relu", bias_grad=True)
    a, b = ref.decode(qdy), ref.decode(qw)
    total, slack, most = (torch.zeros(N, dtype=F64, device="cuda") for _ in range(3))
    for i in range(0, ROWS, 10_000):
        j = min(i + 10_000, ROWS)
        s = (pre[i:j] > 0).to(F64)
        v, off = a[i:j] @ b.t() * s, ref.SUM * (a[i:j].abs() @ b.abs().t()) * s
        ref.close(r.dpre[i:j], v, 1.01 * off + ref.half_step(BF16) * v.abs(), "rows from %d" % i)
        total += v.sum(0)
        slack += off.sum(0)
        most += v.abs().sum(0)
    # additions in fp32: 128 of a thread, then those of the windows (four sums each, an eighth of them in one chain)
    steps = 160 + ROWS // 128
    ref.close(r.dbias, total, 1.01 * (slack + steps * 2.0 ** -24 * most), "dbias")
    assert bsq.device_status() == 0


def test_weight_gradients_pass_32_bits(bsq):
    experts, n, k = 33, 8192, 8192
    counts = [1 + 31 * e % 128 for e in range(experts)]
    c, o, rows, spans = segments(counts, 128)
    live = torch.zeros(rows, 1, dtype=torch.bool, device="cuda")
    for lo, hi in spans:
        live[lo:hi] = True
    qdy = bsq.quantize("mxfp8", (rnd(1, rows, n) * live).to(BF16).t().contiguous())
    qx = bsq.quantize("mxfp8", (rnd(2, rows, k) * live).to(BF16).t().contiguous())
    dw = bsq.expert_gemm_wgrad(qdy, qx, c, o, dtype=F32)
    a, b = ref.decode(qdy), ref.decode(qx)
    for e in (0, 15, 31, 32):  # 2^31 values end inside the 32nd, 2^32 bytes inside the 16th
        lo, hi = spans[e]
        want, size = a[:, lo:hi] @ b[:, lo:hi].t(), a[:, lo:hi].abs() @ b[:, lo:hi].abs().t()
        ref.close(dw[e], want, ref.SUM * size + ref.half_step(F32) * want.abs(), "expert %d" % e)
    assert bsq.device_status() == 0
