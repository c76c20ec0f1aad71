"""Products with activation, residual and their gradients (gemm_act, gemm_act_backward), and the same grouped by
expert (expert_gemm, expert_gemm_backward, expert_gemm_wgrad), against 64 bits."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FORMATS = ["mxfp8", "nvfp4", "mxfp4"]
ACTS = [None, "gelu", "gelu_tanh", "silu", "relu"]


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


def rnd(seed, *shape, std=1.0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) * std


def segments(counts, align=1, behind=0):
    """(counts, offsets, rows, spans): the experts' segments padded to align, `behind` rows of none behind the last."""
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // align) * align)
    spans = [(a, a + c) for a, c in zip(offsets, counts)]
    return (torch.tensor(counts, dtype=torch.int32, device="cuda"), torch.tensor(offsets, dtype=torch.int32, device="cuda"),
            offsets[-1] + behind, spans)


def live_rows(rows, spans):
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a, b in spans:
        live[a:b] = True
    return live


def check_forward(r, a, b, spans, cols, bias, activation, residual, what):
    v, size = ref.sums(a, b, spans, cols)
    live = live_rows(a.shape[0], spans)[:, None]
    if bias is not None:
        per = bias.to(F64).reshape(-1, cols)
        for e, (lo, hi) in enumerate(spans):
            v[lo:hi] += per[e]
    off = ref.SUM * size + 2.0 ** -23 * v.abs()
    if r.pre is not None:
        ref.close(r.pre, v, off + (ref.half_step(BF16) * v.abs()), what + " pre")
    want = torch.where(live, ref.act(activation, v), 0)
    off = 1.13 * off + ref.ACT * v.abs()
    if residual is not None:
        want = want + residual.to(F64)
        off = off + 2.0 ** -23 * want.abs()
    ref.close(r.out, want, off * 1.01 + ref.half_step(r.out.dtype) * want.abs(), what + " out")


def check_backward(r, a, b, spans, cols, pre, activation, what):
    v, size = ref.sums(a, b, spans, cols, stacked_cols=True)
    off = ref.SUM * size
    if pre is not None:
        s = ref.slope(activation, pre.to(F64))
        off = off * s.abs() + ref.ACT * v.abs()
        v = v * s
    live = live_rows(a.shape[0], spans)[:, None]
    v, off = torch.where(live, v, 0), torch.where(live, off, 0)
    ref.close(r.dpre, v, 1.01 * off + ref.half_step(BF16) * v.abs(), what + " dpre")
    if r.dbias is not None:
        want = torch.stack([v[lo:hi].sum(0) for lo, hi in spans])
        # additions in fp32: 128 of a thread, then those of the windows
        steps = 160 + a.shape[0] // 128
        slack = torch.stack([off[lo:hi].sum(0) + steps * 2.0 ** -24 * v[lo:hi].abs().sum(0) for lo, hi in spans])
        ref.close(r.dbias.reshape(want.shape), want, 1.01 * slack, what + " dbias")


# ---------------------------------------------------------------- dense
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,k", [(1, 8, 128), (7, 256, 256), (128, 264, 384), (257, 512, 128), (1001, 1000, 1152)])
def test_dense_product(bsq, fmt, rows, n, k):
    qa, qb = bsq.quantize(fmt, rnd(1, rows, k).to(BF16)), bsq.quantize(fmt, rnd(2, n, k, std=k ** -0.5).to(BF16))
    r = bsq.gemm_act(qa, qb)
    check_forward(r, ref.decode(qa), ref.decode(qb), [(0, rows)], n, None, None, None, "plain")
    assert bsq.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("kind", ["none", "bf16", "fp32", "fp32 out"])
def test_dense_epilogues(bsq, fmt, activation, kind):
    rows, n, k = 333, 392, 256
    qa, qb = bsq.quantize(fmt, rnd(1, rows, k).to(BF16)), bsq.quantize(fmt, rnd(2, n, k, std=2 * k ** -0.5).to(BF16))
    bias = rnd(3, n, std=0.3).to(BF16)
    residual = rnd(4, rows, n + 8).to(F32 if kind == "fp32" else BF16)[:, 8:] if kind in ("bf16", "fp32") else None
    for save_pre in (False, True):
        r = bsq.gemm_act(qa, qb, bias, activation, residual, save_pre, out_dtype=F32 if kind == "fp32 out" else None)
        assert r.out.dtype is (F32 if "fp32" in kind else BF16) and (r.pre is not None) == save_pre
        check_forward(r, ref.decode(qa), ref.decode(qb), [(0, rows)], n, bias, activation, residual, kind)
    assert bsq.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("rows,n,k", [(1, 128, 8), (300, 256, 520), (1027, 384, 256)])
def test_dense_backward(bsq, fmt, activation, rows, n, k):
    qdy = bsq.quantize(fmt, rnd(1, rows, n, std=1e-3).to(BF16))
    qw = bsq.quantize(fmt, rnd(2, k, n, std=n ** -0.5).to(BF16))
    pre = rnd(3, rows, k + 24, std=2.0).to(BF16)[:, 16:16 + k] if activation else None
    for bias_grad in (False, True):
        r = bsq.gemm_act_backward(qdy, qw, pre, activation, bias_grad)
        check_backward(r, ref.decode(qdy), ref.decode(qw), [(0, rows)], k, pre, activation, "dense")
        assert (r.dbias is not None) == bias_grad
    assert bsq.device_status() == 0


# ---------------------------------------------------------------- experts
SEGMENTS = [([5], 1, 0), ([0, 1, 5, 0, 128, 129, 300, 0], 1, 0), ([0, 1, 5, 0, 128, 129, 300, 0], 128, 77),
            ([3, 250, 1, 257, 40, 513], 16, 5), ([0, 0, 0], 1, 40), ([1] * 40, 1, 3), ([700, 2], 512, 0)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,align,behind", SEGMENTS)
@pytest.mark.parametrize("n,k", [(128, 256), (640, 384)])
def test_expert_product(bsq, fmt, counts, align, behind, n, k):
    c, o, rows, spans = segments(counts, align, behind)
    qx = bsq.quantize(fmt, rnd(1, rows, k).to(BF16))
    qw = bsq.quantize(fmt, rnd(2, len(counts) * n, k, std=2 * k ** -0.5).to(BF16))
    bias = rnd(3, len(counts), n, std=0.3).to(BF16)
    a, b = ref.decode(qx), ref.decode(qw)
    out = torch.full((rows, n), float("nan"), device="cuda", dtype=BF16)
    check_forward(bsq.expert_gemm(qx, qw, c, o, out=out), a, b, spans, n, None, None, None, "plain")
    check_forward(bsq.expert_gemm(qx, qw, c, o, bias, "gelu", save_pre=True), a, b, spans, n, bias, "gelu", None, "gelu")
    assert bsq.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,align,behind", SEGMENTS)
def test_expert_backward(bsq, fmt, counts, align, behind):
    n, k = 384, 640
    c, o, rows, spans = segments(counts, align, behind)
    qdy = bsq.quantize(fmt, rnd(1, rows, n, std=1e-3).to(BF16))
    qw = bsq.quantize(fmt, rnd(2, k, len(counts) * n, std=n ** -0.5).to(BF16))
    a, b = ref.decode(qdy), ref.decode(qw)
    check_backward(bsq.expert_gemm_backward(qdy, qw, c, o), a, b, spans, k, None, None, "plain")
    check_backward(bsq.expert_gemm_backward(qdy, qw, c, o, bias_grad=True), a, b, spans, k, None, None, "sums")
    pre = rnd(3, rows, k, std=2.0).to(BF16)
    r = bsq.expert_gemm_backward(qdy, qw, c, o, pre, "silu", bias_grad=True)
    check_backward(r, a, b, spans, k, pre, "silu", "silu")
    assert bsq.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,align,behind", [([5], 128, 0), ([0, 1, 127, 0, 128, 129, 640, 0], 128, 256),
                                                 ([33, 65, 1000], 256, 0), ([0, 0], 128, 128)])
@pytest.mark.parametrize("n,k", [(128, 256), (608, 328)])
def test_expert_weight_gradient(bsq, fmt, dtype, counts, align, behind, n, k):
    c, o, rows, spans = segments(counts, align, behind)
    live = live_rows(rows, spans)
    dy = torch.where(live[:, None], rnd(1, rows, n), 0).to(BF16)
    x = torch.where(live[:, None], rnd(2, rows, k), 0).to(BF16)
    qdy, qx = bsq.quantize(fmt, dy.t().contiguous()), bsq.quantize(fmt, x.t().contiguous())
    dw = bsq.expert_gemm_wgrad(qdy, qx, c, o, dtype=dtype)
    a, b = ref.decode(qdy), ref.decode(qx)
    for e, (lo, hi) in enumerate(spans):
        want, size = a[:, lo:hi] @ b[:, lo:hi].t(), a[:, lo:hi].abs() @ b[:, lo:hi].abs().t()
        ref.close(dw[e], want, ref.SUM * size + ref.half_step(dtype) * want.abs(), "expert %d" % e)
    assert bsq.device_status() == 0


# ---------------------------------------------------------------- few rows, a depth that several pairs share
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows", [1, 8, 31, 32, 33])
@pytest.mark.parametrize("n,k", [(8, 4096), (1000, 2048), (4096, 1024), (4608, 2304), (16384, 512)])
def test_few_rows(bsq, fmt, rows, n, k):
    qa, qb = bsq.quantize(fmt, rnd(1, rows, k).to(BF16)), bsq.quantize(fmt, rnd(2, n, k, std=2 * k ** -0.5).to(BF16))
    a, b, bias = ref.decode(qa), ref.decode(qb), rnd(3, n, std=0.3).to(BF16)
    for activation, residual, dtype in ((None, None, None), ("gelu", None, F32), ("silu", rnd(4, rows, n).to(BF16), None),
                                        (None, rnd(5, rows, n), None)):
        r = bsq.gemm_act(qa, qb, bias, activation, residual, save_pre=True, out_dtype=dtype)
        check_forward(r, a, b, [(0, rows)], n, bias, activation, residual, "few")
    pre = rnd(6, rows, n, std=2.0).to(BF16)
    check_backward(bsq.gemm_act_backward(qa, qb, pre, "gelu", True), a, b, [(0, rows)], n, pre, "gelu", "few")
    assert bsq.device_status() == 0
