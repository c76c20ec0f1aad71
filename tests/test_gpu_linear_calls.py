"""Products with activation, residual and experts: what callers may do with them -- streams, graphs, views, rows of none
that hold anything, segments out of range, many experts, long outputs, stalls -- and both host sides."""
import pytest
import torch

import linear_ref as ref
from test_gpu_host_paths import both, same
from test_gpu_linear import check_backward, check_forward, live_rows, rnd, segments

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture()
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


def operands(bsq, fmt, rows, n, k, experts=1, seed=1):
    return (bsq.quantize(fmt, rnd(seed, rows, k).to(BF16)),
            bsq.quantize(fmt, rnd(seed + 1, experts * n, k, std=2 * k ** -0.5).to(BF16)))


def test_both_host_sides_give_the_same(bsq, monkeypatch):
    qx, qw = operands(bsq, "nvfp4", 333, 256, 384)
    bias, res = rnd(3, 256).to(BF16), rnd(4, 333, 264).to(BF16)[:, :256]
    c, o, rows, _ = segments([5, 0, 200, 128], 1)
    ex, ew = operands(bsq, "nvfp4", rows, 256, 384, 4)
    dy, wc = bsq.quantize("nvfp4", rnd(5, rows, 256).to(BF16)), bsq.quantize("nvfp4", rnd(6, 384, 1024).to(BF16))
    wc1 = bsq.quantize("nvfp4", rnd(6, 384, 256).to(BF16))
    pre = rnd(7, rows, 384).to(BF16)
    c2, o2, rows2, _ = segments([5, 0, 200, 128], 128)
    yc, xc = (bsq.quantize("nvfp4", rnd(s, m, rows2).to(BF16)) for s, m in ((8, 128), (9, 256)))
    for call in (lambda: bsq.gemm_act(qx, qw, bias, "gelu", res, True),
                 lambda: bsq.gemm_act(qx, qw, out_dtype=F32), lambda: bsq.gemm_act(qx, qw, None, "relu", res.float()),
                 lambda: bsq.expert_gemm(ex, ew, c, o, bias.expand(4, 256).contiguous(), "silu", True),
                 lambda: bsq.gemm_act_backward(dy, wc1, pre, "gelu_tanh", True), lambda: bsq.gemm_act_backward(dy, wc1),
                 lambda: bsq.expert_gemm_backward(dy, wc, c, o, pre, "gelu", True),
                 lambda: bsq.expert_gemm_wgrad(yc, xc, c2, o2), lambda: bsq.expert_gemm_wgrad(yc, xc, c2, o2, dtype=F32)):
        a, b = both(bsq, monkeypatch, call)
        same(a, b)
    assert bsq.device_status() == 0


def test_refusals(bsq):
    qx, qw = operands(bsq, "mxfp8", 16, 128, 128)
    r = torch.zeros(16, 132, device="cuda", dtype=BF16)
    for residual in (r[:, 1:129], r[:, :128]):  # an odd address; rows of no whole vectors
        with pytest.raises(bsq.BsqError) as e:
            bsq.gemm_act(qx, qw, residual=residual)
        assert e.value.code == bsq.ERR_ALIGN
    with pytest.raises(AssertionError):
        bsq.gemm_act(qx, qw, residual=r[:8, :128])
    with pytest.raises(AssertionError):
        bsq.gemm_act(qx, qw, torch.zeros(127, device="cuda", dtype=BF16))
    with pytest.raises(TypeError):
        bsq.gemm_act(qx, qw, torch.zeros(128, device="cuda"))
    with pytest.raises(AssertionError):
        bsq.gemm_act(bsq.QTensor(qx.fmt, 17, 128, qx.codes, qx.scales), qw)  # codes of 16 rows
    c, o, _, _ = segments([8, 8])
    with pytest.raises(AssertionError):
        bsq.expert_gemm(qx, qw, c, o[:2])
    with pytest.raises(bsq.BsqError) as e:  # 64 columns an expert: not whole scale tiles
        bsq.expert_gemm(qx, qw, c, o)
    assert e.value.code == bsq.ERR_SHAPE
    with pytest.raises(AssertionError):
        bsq.gemm_act_backward(qx, qw, activation="gelu")
    with pytest.raises(AssertionError):
        bsq.gemm_act_backward(qx, qw, torch.zeros(16, 128, device="cuda", dtype=BF16))


def test_no_rows(bsq):
    _, qw = operands(bsq, "mxfp4", 1, 256, 128)
    q0 = bsq.empty_qtensor("mxfp4", 0, 128)
    r = bsq.gemm_act(q0, qw, activation="gelu", save_pre=True)
    assert r.out.shape == r.pre.shape == (0, 256)
    g = bsq.gemm_act_backward(q0, qw, bias_grad=True)
    assert g.dpre.shape == (0, 256) and not g.dbias.any()
    c, o, _, _ = segments([0, 0])
    e = bsq.expert_gemm_backward(q0, bsq.quantize("mxfp4", rnd(1, 128, 256).to(BF16)), c, o, bias_grad=True)
    assert e.dpre.shape == (0, 128) and e.dbias.shape == (2, 128) and not e.dbias.any()
    w = bsq.expert_gemm_wgrad(bsq.empty_qtensor("mxfp4", 128, 0), bsq.empty_qtensor("mxfp4", 64, 0), c, o)
    assert w.shape == (2, 128, 64) and not w.any()


@pytest.mark.parametrize("align", [1, 128])
def test_rows_of_none_may_hold_nan(bsq, align):
    """NaN codes and scales in rows of none, and NaN in their kept arguments, reach no result."""
    counts = [3, 0, 130, 61]
    c, o, rows, spans = segments(counts, align, 70)
    none = ~live_rows(rows, spans)
    qx, qw = operands(bsq, "mxfp8", rows, 256, 128, 4)
    a, b = ref.decode(qx), ref.decode(qw)
    qx.codes.view(rows, 128)[none] = 0x7F
    r = torch.arange(rows, device="cuda")[none]
    for col in range(4):
        qx.scales[(r // 128) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4 + col] = 0xFF
    check_forward(bsq.expert_gemm(qx, qw, c, o, None, "gelu", True), a, b, spans, 256, None, "gelu", None, "nan rows")
    wc = bsq.quantize("mxfp8", rnd(5, 384, 4 * 128).to(BF16))
    pre = rnd(6, rows, 384).to(BF16)
    pre[none] = float("nan")
    g = bsq.expert_gemm_backward(qx, wc, c, o, pre, "gelu", bias_grad=True)
    check_backward(g, a, ref.decode(wc), spans, 384, torch.nan_to_num(pre), "gelu", "nan rows")
    assert bsq.device_status() == 0


def test_nan_and_infinity_stay_where_they_are(bsq):
    """An argument that is NaN or infinite touches its own gradient alone; the residual's its own output."""
    qdy, qw = operands(bsq, "mxfp8", 200, 256, 128)
    clean = rnd(3, 200, 256).to(BF16)
    for act in ("gelu", "gelu_tanh", "silu", "relu"):
        pre = clean.clone()
        pre[7, 9], pre[8, 9], pre[100, 31] = float("nan"), float("inf"), -0.0
        a = bsq.gemm_act_backward(qdy, qw, clean, act).dpre
        b = bsq.gemm_act_backward(qdy, qw, pre, act).dpre
        other = torch.ones_like(a, dtype=torch.bool)
        other[7, 9] = other[8, 9] = other[100, 31] = False
        assert torch.equal(a[other], b[other])
        assert act == "relu" or torch.isnan(b[7, 9])
        v = bsq.gemm_act_backward(qdy, qw).dpre[100, 31].float()
        want = 0.0 if act == "relu" else 0.5
        assert abs(float(b[100, 31]) - want * float(v)) <= 2 ** -7 * abs(float(v))
    res = clean.clone()
    res[3, 5] = float("inf")
    a, b = bsq.gemm_act(qdy, qw, residual=clean).out, bsq.gemm_act(qdy, qw, residual=res).out
    assert torch.isinf(b[3, 5]) and int((a != b).sum()) == 1


def test_one_row_of_a_wider_matrix(bsq):
    """A single row's stride says nothing: any will do."""
    qx, qw = operands(bsq, "mxfp8", 1, 128, 256)
    wide = rnd(3, 8, 131).to(BF16)
    row = wide.view(-1)[:128].as_strided((1, 128), (131, 1))
    assert torch.equal(bsq.gemm_act(qx, qw, residual=row).out, bsq.gemm_act(qx, qw, residual=row.clone()).out)
    g = [bsq.gemm_act_backward(qx, qw, p, "gelu").dpre for p in (row, row.clone())]
    assert torch.equal(*g)


def test_segments_that_overlap_stay_within_the_workspace(bsq):
    """Not a call with a result; nothing is written past what the call was given."""
    t = dict(dtype=torch.int32, device="cuda")
    experts, rows, n = 64, 600, 128
    qdy, qw = bsq.quantize("mxfp8", rnd(1, rows, n).to(BF16)), bsq.quantize("mxfp8", rnd(2, 256, experts * n).to(BF16))
    counts = torch.full((experts,), rows, **t)
    offsets = torch.tensor([0, rows] * (experts // 2) + [0], **t)
    nbytes = bsq.bsq_gemm_act_backward_workspace(rows, 256, experts)
    ws = torch.full((nbytes + 4096,), 7, dtype=torch.uint8, device="cuda")
    out = torch.empty(rows, 256, dtype=BF16, device="cuda")
    dbias = torch.empty(experts, 256, device="cuda")
    a = bsq.LinearArgs(fmt=bsq.MXFP8, flags=bsq.FLAG_STACK_COLS, rows=rows, cols=256, depth=n, experts=experts,
                       A=qdy.codes.data_ptr(), A_scales=qdy.scales.data_ptr(), B=qw.codes.data_ptr(),
                       B_scales=qw.scales.data_ptr(), counts=counts.data_ptr(), offsets=offsets.data_ptr(),
                       out=out.data_ptr(), dbias=dbias.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=nbytes)
    assert bsq.bsq_gemm_act_backward(a) == bsq.OK and bsq.device_status() == 0
    assert bool((ws[nbytes:] == 7).all())


def test_the_residual_may_be_the_output(bsq):
    for dtype in (BF16, F32):
        qx, qw = operands(bsq, "mxfp4", 777, 512, 256)
        res = rnd(3, 777, 512).to(dtype)
        want = bsq.gemm_act(qx, qw, None, "gelu", res).out
        got = bsq.gemm_act(qx, qw, None, "gelu", res, out=res)
        assert got.out is res and torch.equal(res, want)


def test_segments_out_of_range_are_taken_as_the_nearest_in_range(bsq):
    n, k = 256, 128
    qx, qw = operands(bsq, "mxfp8", 300, n, k, 3)
    a, b = ref.decode(qx), ref.decode(qw)

    def run(counts, offsets):
        t = dict(dtype=torch.int32, device="cuda")
        return bsq.expert_gemm(qx, qw, torch.tensor(counts, **t), torch.tensor(offsets, **t))

    for counts, offsets, spans in [
            ([10, 2 ** 31 - 1, 0], [0, 10, 2 ** 31 - 1, 2 ** 31 - 1], [(0, 10), (10, 300), (300, 300)]),
            ([-5, 20, 30], [-7, 50, 100, 130], [(0, 0), (50, 70), (100, 130)]),
            ([40, 5, 5], [0, 20, 200, 100], [(0, 20), (20, 25), (200, 200)])]:
        check_forward(run(counts, offsets), a, b, spans, n, None, None, None, str(offsets))
    assert bsq.device_status() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "mxfp4"])
def test_weight_gradient_of_segments_that_begin_inside_a_tile(bsq, fmt):
    """No address that the tensor copies cannot take: zeros for that expert, and the status says so."""
    t = dict(dtype=torch.int32, device="cuda")
    qdy, qx = bsq.quantize(fmt, rnd(1, 128, 512).to(BF16)), bsq.quantize(fmt, rnd(2, 64, 512).to(BF16))
    counts, offsets = torch.tensor([100, 60, 128], **t), torch.tensor([0, 129, 384, 512], **t)
    dw = bsq.expert_gemm_wgrad(qdy, qx, counts, offsets)
    assert bsq.device_status() == bsq.ERR_SHAPE and bsq.device_status() == 0
    a, b = ref.decode(qdy), ref.decode(qx)
    assert not dw[1].any()
    want, size = a[:, 384:] @ b[:, 384:].t(), a[:, 384:].abs() @ b[:, 384:].abs().t()
    ref.close(dw[2], want, ref.SUM * size + ref.half_step(BF16) * want.abs())
    # out of range: nothing is read past the operands
    dw = bsq.expert_gemm_wgrad(qdy, qx, torch.tensor([2 ** 31 - 1, 5, -3], **t), torch.tensor([256, 2 ** 31 - 1, -128, 0], **t))
    want, size = a[:, 256:] @ b[:, 256:].t(), a[:, 256:].abs() @ b[:, 256:].abs().t()
    ref.close(dw[0], want, ref.SUM * size + ref.half_step(BF16) * want.abs())
    assert not dw[1:].any() and bsq.device_status() == 0


@pytest.mark.parametrize("experts", [1, 300, 2048])
def test_many_experts(bsq, experts):
    g = torch.Generator().manual_seed(experts)
    counts = torch.randint(0, 4, (experts,), generator=g).tolist()
    counts[0], counts[-1] = 2, 3
    c, o, rows, spans = segments(counts, 1, 9)
    qx, qw = operands(bsq, "mxfp4", rows, 128, 128, experts)
    check_forward(bsq.expert_gemm(qx, qw, c, o), ref.decode(qx), ref.decode(qw), spans, 128, None, None, None, "many")
    c, o, rows, spans = segments(counts, 128)
    live = live_rows(rows, spans)[:, None]
    dy, x = (torch.where(live, rnd(s, rows, 128), 0).to(BF16) for s in (1, 2))
    qdy, qx = bsq.quantize("mxfp4", dy.t().contiguous()), bsq.quantize("mxfp4", x.t().contiguous())
    dw, a, b = bsq.expert_gemm_wgrad(qdy, qx, c, o, dtype=F32), ref.decode(qdy), ref.decode(qx)
    for e in {0, experts // 2, experts - 1}:
        lo, hi = spans[e]
        want, size = a[:, lo:hi] @ b[:, lo:hi].t(), a[:, lo:hi].abs() @ b[:, lo:hi].abs().t()
        ref.close(dw[e], want, ref.SUM * size + ref.half_step(F32) * want.abs(), "expert %d" % e)
    assert bsq.device_status() == 0


def test_outputs_whose_offsets_pass_32_bits(bsq):
    rows, n, k = 270_001, 8192, 128
    x = rnd(1, rows, k).to(BF16)
    qx, qw = bsq.quantize("mxfp8", x), bsq.quantize("mxfp8", rnd(2, n, k, std=0.1).to(BF16))
    c, o, _, _ = segments([5, rows - 9, 4])
    e = bsq.quantize("mxfp8", rnd(3, 3 * n, k, std=0.1).to(BF16))
    a, b, w = ref.decode(qx), ref.decode(qw), ref.decode(e)
    pick = torch.cat([torch.arange(0, 300), torch.arange(262_100, 262_200), torch.arange(rows - 300, rows)]).cuda()
    expert = torch.where(pick < 5, 0, torch.where(pick < rows - 4, 1, 2))
    dense, grouped = bsq.gemm_act(qx, qw).out, bsq.expert_gemm(qx, e, c, o).out
    tol = lambda v, s: ref.SUM * s + ref.half_step(BF16) * v.abs()  # noqa: E731
    v, s = a[pick] @ b.t(), a[pick].abs() @ b.abs().t()
    ref.close(dense[pick], v, tol(v, s))
    for i in range(3):
        at = pick[expert == i]
        v, s = a[at] @ w[i * n:(i + 1) * n].t(), a[at].abs() @ w[i * n:(i + 1) * n].abs().t()
        ref.close(grouped[at], v, tol(v, s), "expert %d" % i)
    assert bsq.device_status() == 0


def test_the_same_inputs_give_the_same_bits(bsq):
    c, o, rows, _ = segments([700, 0, 33, 1500, 129], 128, 128)
    dy, wc = bsq.quantize("mxfp8", rnd(1, rows, 256).to(BF16)), bsq.quantize("mxfp8", rnd(2, 384, 5 * 256).to(BF16))
    pre = rnd(3, rows, 384).to(BF16)
    first = bsq.expert_gemm_backward(dy, wc, c, o, pre, "gelu", bias_grad=True)
    for _ in range(20):
        again = bsq.expert_gemm_backward(dy, wc, c, o, pre, "gelu", bias_grad=True)
        assert torch.equal(again.dpre, first.dpre) and torch.equal(again.dbias, first.dbias)


def test_calls_run_on_the_stream_that_they_are_given(bsq):
    rows, n, k = 4000, 512, 512
    x, w = rnd(1, rows, k).to(BF16), rnd(2, n, k, std=0.05).to(BF16)
    want = bsq.gemm_act(bsq.quantize("mxfp4", x), bsq.quantize("mxfp4", w), None, "gelu", save_pre=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, kept = [], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)  # the operands come late
            late = x + 0
        qx = bsq.quantize("mxfp4", late, stream=s)
        qw = bsq.quantize("mxfp4", w, stream=s)
        # quantize allocates on the current stream: what stream s still reads must not be given back to it
        kept += [late, qx, qw]
        got.append(bsq.gemm_act(qx, qw, None, "gelu", save_pre=True, stream=s))
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r.out, want.out) and torch.equal(r.pre, want.pre)


def test_a_captured_graph_follows_the_segments(bsq):
    """Sort, gather, quantize, product, weighted sum in one graph: replayed on other choices of experts it gives what
    eager calls give."""
    tokens, topk, experts, k, n = 300, 2, 8, 256, 256
    x = rnd(1, tokens, k).to(BF16)
    qw = bsq.quantize("mxfp8", rnd(2, experts * n, k, std=0.1).to(BF16))
    ids = torch.zeros(tokens, topk, device="cuda", dtype=torch.int64)
    weights = torch.rand(tokens, topk, device="cuda")

    def chain():
        s = bsq.expert_sort(ids, experts, align=1)
        q = bsq.quantize("mxfp8", bsq.expert_gather(x, s.position, s.slot))
        return bsq.expert_combine(bsq.expert_gemm(q, qw, s.counts, s.offsets, activation="silu").out, s.position, weights)

    def choices(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        c = torch.rand(tokens, experts, device="cuda", generator=g).topk(topk, dim=-1).indices
        c[torch.rand(tokens, topk, device="cuda", generator=g) < 0.1] = -1  # dropped
        return c

    ids.copy_(choices(0))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        chain()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = chain()
    torch.cuda.synchronize()
    for seed in range(1, 5):
        ids.copy_(choices(seed))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, chain())
    assert bsq.device_status() == 0


def test_experts_against_one_product_each(bsq):
    """The grouped product gives the bits of the plain GEMM's operands one expert at a time, within its rounding."""
    counts = [200, 0, 129, 64]
    c, o, rows, spans = segments(counts, 128)
    n, k = 256, 256
    x, w = rnd(1, rows, k).to(BF16), rnd(2, 4 * n, k, std=0.1).to(BF16)
    out = bsq.expert_gemm(bsq.quantize("mxfp8", x), bsq.quantize("mxfp8", w), c, o).out
    for e, (lo, hi) in enumerate(spans):
        if hi > lo:
            one = bsq.gemm(bsq.quantize("mxfp8", x[lo:hi].contiguous()), bsq.quantize("mxfp8", w[e * n:(e + 1) * n].contiguous()))
            err = (one.double() - out[lo:hi].double()).abs()
            assert bool((err <= 2 ** -7 * one.double().abs() + 1e-4).all())


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,after", [(600, 0), (600, 1), (600, 7), (16, 0), (16, 1)])
def test_a_stalled_load_gives_up_and_says_so(bsq, fmt, rows, after):
    """Of one window after another, and of few rows, where several pairs wait for each other's sums as well."""
    import time

    qx, qw = operands(bsq, fmt, rows, 512, 2048)
    pre = rnd(3, rows, 512).to(BF16)
    want = bsq.gemm_act(qx, qw, None, "gelu", pre)
    grad = bsq.gemm_act_backward(qx, qw, pre, "gelu", True)
    torch.cuda.synchronize()
    for call in (lambda: bsq.gemm_act(qx, qw, None, "gelu", pre), lambda: bsq.gemm_act_backward(qx, qw, pre, "gelu", True)):
        assert bsq.bsq_test_inject_stall(bsq.KERNEL_LINEAR, after, 2_000_000) == bsq.OK
        t = time.time()
        call()
        assert bsq.device_status() == bsq.ERR_TIMEOUT and time.time() - t < 2.0
    again = bsq.gemm_act(qx, qw, None, "gelu", pre)
    assert torch.equal(again.out, want.out) and bsq.device_status() == 0
    g = bsq.gemm_act_backward(qx, qw, pre, "gelu", True)
    assert torch.equal(g.dpre, grad.dpre) and torch.equal(g.dbias, grad.dbias) and bsq.device_status() == 0


def test_a_stall_behind_the_last_stage_changes_nothing(bsq):
    qx, qw = operands(bsq, "mxfp8", 100, 256, 256)
    want = bsq.gemm_act(qx, qw)
    assert bsq.bsq_test_inject_stall(bsq.KERNEL_LINEAR, 1 << 40, 1_000_000_000) == bsq.OK
    assert torch.equal(bsq.gemm_act(qx, qw).out, want.out) and bsq.device_status() == 0


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu", "relu"])
def test_the_kept_argument_gives_the_derivative(bsq, activation):
    """The derivative that the backward pass multiplies by against differences of the forward's activation, over the whole
    range: the product is 1 (an identity weight), so dpre is act' of the kept argument itself."""
    k = 128
    eye = bsq.quantize("mxfp8", torch.eye(k, device="cuda").to(BF16))
    ones = bsq.quantize("mxfp8", torch.ones(512, k, device="cuda").to(BF16))
    pre = torch.linspace(-9, 9, 512 * k, device="cuda").reshape(512, k).to(BF16)
    got = bsq.gemm_act_backward(ones, eye, pre, activation).dpre.double()
    x, h = pre.double(), 1e-5
    want = (ref.act(activation, x + h) - ref.act(activation, x - h)) / (2 * h)
    away = (x.abs() > 1e-4) | (activation != "relu")  # relu's kink
    # half a bf16 step, the fp32 evaluation, and the differences' own error (h^2 and 1e-16 / h)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 + 1e-9
    assert bool(((got - want).abs() <= tol)[away].all())
