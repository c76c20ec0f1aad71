"""The experts' weight gradients where segments, and the operands, end elsewhere than at a multiple of 128: inside a group
of scales, and with the 4-bit formats inside a step of the depth (64 rows)."""
import pytest
import torch

import linear_ref as ref
from test_gpu_linear import live_rows, rnd

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FORMATS = ["mxfp8", "nvfp4", "mxfp4"]
STEP = {"mxfp8": 32, "nvfp4": 64, "mxfp4": 64}  # rows that one instruction sums over


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


def of(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def operands(bsq, fmt, n, k, rows, zero=None):
    dy, x = rnd(1, rows, n), rnd(2, rows, k)
    if zero is not None:
        dy[zero], x[zero] = 0, 0
    return bsq.quantize(fmt, dy.to(BF16).t().contiguous()), bsq.quantize(fmt, x.to(BF16).t().contiguous())


def check(dw, a, b, spans, dtype):
    """spans: an expert's rows, or None where zeros are due."""
    for e, span in enumerate(spans):
        if span is None:
            assert not dw[e].any(), "expert %d" % e
            continue
        lo, hi = span
        want, size = a[:, lo:hi] @ b[:, lo:hi].t(), a[:, lo:hi].abs() @ b[:, lo:hi].abs().t()
        ref.close(dw[e], want, ref.SUM * size + ref.half_step(dtype) * want.abs(), "expert %d" % e)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,counts,offsets", [
    (32, [32], [0, 32]), (32, [5], [0, 32]), (160, [128, 32], [0, 128, 160]), (160, [100, 1], [0, 128, 160]),
    (224, [128, 96], [0, 128, 224]), (224, [0, 90], [0, 128, 224]), (224, [224], [0, 224]), (96, [96, 0], [0, 96, 96])])
def test_operands_that_end_inside_a_group_of_scales(bsq, fmt, dtype, rows, counts, offsets):
    spans = [(a, a + c) for a, c in zip(offsets, counts)]
    qdy, qx = operands(bsq, fmt, 136, 72, rows, ~live_rows(rows, spans))
    dw = bsq.expert_gemm_wgrad(qdy, qx, of(counts), of(offsets), dtype=dtype)
    check(dw, ref.decode(qdy), ref.decode(qx), spans, dtype)
    assert bsq.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,offsets", [
    ([128, 32], [0, 128, 160]),        # the last segment ends ahead of the operands, between 4-bit steps
    ([128, 33], [0, 128, 161]),        # and inside a step of any format
    ([129, 100], [0, 129, 256]),       # a segment ends inside a step, and the next begins there
    ([64, 100], [0, 65, 256]),         # whole steps: only the next is refused
    ([64, 0], [0, 64, 64]), ([1, 0], [0, 1, 1]), ([300, 2], [0, 200, 2 ** 31 - 1])])
def test_no_expert_takes_in_rows_behind_its_segment(bsq, fmt, counts, offsets):
    """All rows hold values. What one step of the depth would take in from behind a segment is no part of its sum: right,
    or zeros and the status."""
    rows, step = 256, STEP[fmt]
    qdy, qx = operands(bsq, fmt, 128, 64, rows)
    spans, refused = [], False
    for e, c in enumerate(counts):
        lo, end = min(offsets[e], rows), min(offsets[e + 1], rows)
        c = min(c, end - lo)
        past = lo + -(-c // step) * step > end and end < rows
        refused |= c > 0 and (lo % 128 != 0 or past)
        # rows behind the count, up to the step's end, belong to the segment and are not zeros here: not compared
        inside = c % step == 0 or lo + c == rows
        spans.append(None if c == 0 or lo % 128 or past else (lo, lo + c) if inside else "skip")
    dw = bsq.expert_gemm_wgrad(qdy, qx, of(counts), of(offsets))
    a, b = ref.decode(qdy), ref.decode(qx)
    keep = [e for e, s in enumerate(spans) if s != "skip"]
    check(dw[keep], a, b, [spans[e] for e in keep], BF16)
    assert bsq.device_status() == (bsq.ERR_SHAPE if refused else 0) and bsq.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_the_experts_beside_a_refused_one_keep_their_gradients(bsq, fmt):
    counts, offsets = [100, 60, 128], [0, 129, 384, 512]
    zero = ~live_rows(512, [(0, 100), (129, 189), (384, 512)])
    qdy, qx = operands(bsq, fmt, 128, 64, 512, zero)
    dw = bsq.expert_gemm_wgrad(qdy, qx, of(counts), of(offsets))
    assert bsq.device_status() == bsq.ERR_SHAPE and bsq.device_status() == 0
    check(dw, ref.decode(qdy), ref.decode(qx), [(0, 100), None, (384, 512)], BF16)
