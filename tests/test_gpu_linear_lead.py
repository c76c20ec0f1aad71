"""Products of experts whose first segment does not begin at row 0: the rows ahead of it are rows of none, zeros in every
output, whatever stood there."""
import pytest
import torch

import linear_ref as ref
from test_gpu_linear import check_backward, check_forward, rnd

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
ROWS = 600
# counts, offsets, the rows that they stand for
LEADS = [([40, 60], [5, 100, 200], [(5, 45), (100, 160)]),
         ([72, 0, 100], [128, 200, 200, 300], [(128, 200), (200, 200), (200, 300)]),
         ([10], [257, 300], [(257, 267)]),
         ([88, 1], [511, 599, 600], [(511, 599), (599, 600)]),
         ([7, 7], [600, 600, 600], [(600, 600), (600, 600)]),
         ([7, 7], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [(600, 600), (600, 600)]),
         # offsets that fall: the rows ahead are those ahead of every segment
         ([9, 50, 30], [300, 20, 100, 200], [(300, 300), (20, 70), (100, 130)])]


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


def of(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def stale(rows, cols):
    return torch.full((rows, cols), float("nan"), device="cuda", dtype=BF16)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,offsets,spans", LEADS)
def test_rows_ahead_of_the_first_segment_are_zeros(bsq, fmt, counts, offsets, spans):
    n, k, experts = 256, 384, len(counts)
    c, o = of(counts), of(offsets)
    qx = bsq.quantize(fmt, rnd(1, ROWS, k).to(BF16))
    qw = bsq.quantize(fmt, rnd(2, experts * n, k, std=2 * k ** -0.5).to(BF16))
    bias = rnd(3, experts, n, std=0.3).to(BF16)
    a, b = ref.decode(qx), ref.decode(qw)
    check_forward(bsq.expert_gemm(qx, qw, c, o, out=stale(ROWS, n)), a, b, spans, n, None, None, None, "plain")
    r = bsq.GemmAct(stale(ROWS, n), stale(ROWS, n))
    args = bsq.LinearArgs(fmt=qx.fmt, activation=bsq.ACTIVATIONS["gelu"], rows=ROWS, cols=n, depth=k, experts=experts,
                          A=qx.codes.data_ptr(), A_scales=qx.scales.data_ptr(), B=qw.codes.data_ptr(),
                          B_scales=qw.scales.data_ptr(), counts=c.data_ptr(), offsets=o.data_ptr(), bias=bias.data_ptr(),
                          out=r.out.data_ptr(), pre=r.pre.data_ptr())
    assert bsq.bsq_gemm_act(args) == bsq.OK
    check_forward(r, a, b, spans, n, bias, "gelu", None, "gelu")
    assert bsq.device_status() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,offsets,spans", LEADS)
def test_their_gradients_are_zeros(bsq, fmt, counts, offsets, spans):
    n, k, experts = 384, 640, len(counts)
    c, o = of(counts), of(offsets)
    qdy = bsq.quantize(fmt, rnd(1, ROWS, n, std=1e-3).to(BF16))
    qw = bsq.quantize(fmt, rnd(2, k, experts * n, std=n ** -0.5).to(BF16))
    a, b = ref.decode(qdy), ref.decode(qw)
    pre = rnd(3, ROWS, k, std=2.0).to(BF16)
    for kept, activation, sums in ((None, None, False), (None, None, True), (pre, "silu", True)):
        r = bsq.expert_gemm_backward(qdy, qw, c, o, kept, activation, bias_grad=sums, out=stale(ROWS, k))
        check_backward(r, a, b, spans, k, kept, activation, "lead")
    assert bsq.device_status() == 0


def test_what_stands_ahead_is_not_read(bsq):
    """NaN codes and kept arguments ahead of the first segment reach nothing."""
    counts, offsets, spans = [40, 60], [150, 200, 300], [(150, 190), (200, 260)]
    qx = bsq.quantize("mxfp8", rnd(1, ROWS, 128).to(BF16))
    qw = bsq.quantize("mxfp8", rnd(2, 128, 2 * 128).to(BF16))
    a, b = ref.decode(qx), ref.decode(qw)
    a[:150] = 0
    qx.codes.view(ROWS, 128)[:150] = 0x7F
    pre = rnd(3, ROWS, 128).to(BF16)
    pre[:150] = float("nan")
    r = bsq.expert_gemm_backward(qx, qw, of(counts), of(offsets), pre, "gelu", bias_grad=True, out=stale(ROWS, 128))
    check_backward(r, a, b, spans, 128, torch.nan_to_num(pre), "gelu", "nan ahead")
    assert bsq.device_status() == 0


def test_many_experts_behind_a_long_lead(bsq):
    experts, lead, n, k = 2048, 1000, 128, 128
    counts = [1 + (e % 3 == 0) for e in range(experts)]
    offsets = [lead]
    for e in range(experts):
        offsets.append(offsets[-1] + 2)
    spans = [(x, x + m) for x, m in zip(offsets, counts)]
    rows = offsets[-1] + 77
    qx = bsq.quantize("mxfp4", rnd(1, rows, k).to(BF16))
    qw = bsq.quantize("mxfp4", rnd(2, experts * n, k, std=k ** -0.5).to(BF16))
    r = bsq.expert_gemm(qx, qw, of(counts), of(offsets), out=stale(rows, n))
    check_forward(r, ref.decode(qx), ref.decode(qw), spans, n, None, None, None, "many")
    assert bsq.device_status() == 0
