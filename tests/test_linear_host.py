"""Host-side checks of the products with activation, residual and experts: refusals before any CUDA call."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


P = 1 << 20  # an aligned address that is never dereferenced


def args(bsq, **kw):
    a = bsq.LinearArgs()
    for k, v in dict(dict(fmt=bsq.MXFP8, rows=4, cols=128, depth=256, A=P, A_scales=P, B=P, B_scales=P, out=P), **kw).items():
        setattr(a, k, v)
    return a


def test_sizes_of_the_structure(bsq):
    assert ctypes.sizeof(bsq.LinearArgs) == bsq._LINEAR_ARGS.size


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=7), "ERR_ARG"), (dict(flags=0x100), "ERR_ARG"), (dict(rows=-1), "ERR_ARG"), (dict(cols=0), "ERR_ARG"),
    (dict(depth=0), "ERR_ARG"), (dict(A=None), "ERR_ARG"), (dict(B_scales=None), "ERR_ARG"), (dict(out=None), "ERR_ARG"),
    (dict(activation=5), "ERR_ARG"), (dict(activation=-1), "ERR_ARG"), (dict(experts=-1), "ERR_ARG"),
    (dict(experts=2), "ERR_ARG"), (dict(experts=2, counts=P, offsets=None), "ERR_ARG"),
    (dict(grad_pre=P, grad_pre_stride=128), "ERR_ARG"), (dict(dbias=P), "ERR_ARG"),
    (dict(experts=2, counts=P, offsets=P, residual=P, residual_stride=128), "ERR_ARG"),
    (dict(depth=64), "ERR_SHAPE"), (dict(depth=192), "ERR_SHAPE"), (dict(cols=12), "ERR_SHAPE"),
    (dict(rows=1 << 31), "ERR_SHAPE"), (dict(cols=1 << 31), "ERR_SHAPE"),
    (dict(experts=2, counts=P, offsets=P, cols=136), "ERR_SHAPE"),
    (dict(experts=2049, counts=P, offsets=P), "ERR_SHAPE"),
    (dict(experts=2048, counts=P, offsets=P, cols=1 << 20), "ERR_SHAPE"),
    (dict(residual=P, residual_stride=127), "ERR_SHAPE"), (dict(residual=P, residual_stride=0), "ERR_SHAPE"),
    (dict(residual=P, residual_stride=129), "ERR_ALIGN"), (dict(residual=P + 2, residual_stride=128), "ERR_ALIGN"),
    (dict(A=P + 8), "ERR_ALIGN"), (dict(out=P + 2), "ERR_ALIGN"), (dict(pre=P + 4), "ERR_ALIGN"), (dict(bias=P + 1), "ERR_ALIGN"),
    (dict(experts=2, counts=P + 2, offsets=P), "ERR_ALIGN")])
def test_forward_refusals(bsq, kw, code):
    assert bsq.bsq_gemm_act(args(bsq, **kw)) == getattr(bsq, code)


@pytest.mark.parametrize("kw,code", [
    (dict(bias=P), "ERR_ARG"), (dict(residual=P, residual_stride=128), "ERR_ARG"), (dict(pre=P), "ERR_ARG"),
    (dict(flags=0x4000), "ERR_ARG"), (dict(activation=1), "ERR_ARG"), (dict(grad_pre=P, grad_pre_stride=128), "ERR_ARG"),
    (dict(activation=1, grad_pre=P, grad_pre_stride=120), "ERR_SHAPE"),
    (dict(activation=1, grad_pre=P, grad_pre_stride=132), "ERR_ALIGN"),
    (dict(dbias=P + 2), "ERR_ALIGN"), (dict(dbias=P), "ERR_ARG"), (dict(dbias=P, workspace=P, workspace_bytes=16), "ERR_ARG"),
    (dict(dbias=P, workspace=P + 8, workspace_bytes=1 << 20), "ERR_ALIGN")])
def test_backward_refusals(bsq, kw, code):
    assert bsq.bsq_gemm_act_backward(args(bsq, **kw)) == getattr(bsq, code)


def test_weight_gradient_refusals(bsq):
    def call(fmt=bsq.MXFP4, dy=P, x=P, counts=P, offsets=P, rows=256, N=128, K=128, experts=2, out=P):
        return bsq.bsq_expert_gemm_wgrad(fmt, dy, P, x, P, counts, offsets, rows, N, K, experts, out)

    assert call(fmt=9) == bsq.ERR_ARG and call(fmt=bsq.MXFP4 | 0x100) == bsq.ERR_ARG
    assert call(experts=0) == bsq.ERR_ARG and call(counts=None) == bsq.ERR_ARG and call(out=None) == bsq.ERR_ARG
    assert call(N=0) == bsq.ERR_ARG and call(rows=-1) == bsq.ERR_ARG and call(dy=None) == bsq.ERR_ARG
    assert call(K=12) == bsq.ERR_SHAPE and call(rows=48) == bsq.ERR_SHAPE and call(experts=2049) == bsq.ERR_SHAPE
    assert call(N=1 << 30, experts=2) == bsq.ERR_SHAPE
    assert call(dy=P + 8) == bsq.ERR_ALIGN and call(offsets=P + 2) == bsq.ERR_ALIGN


def test_workspace_sizes(bsq):
    ws = bsq.bsq_gemm_act_backward_workspace
    assert ws(-1, 128) == 0 and ws(4, 0) == 0 and ws(4, 128, -1) == 0 and ws(4, 128, 4096) == 0
    assert ws(1, 128) >= 128 * 4 and ws(1, 128, 4) > ws(1, 128) and ws(100000, 128) >= 390 * 128 * 4


def test_a_valid_call_reaches_the_device_check(bsq):
    if torch.cuda.is_available():
        pytest.skip("a device is there")
    assert bsq.bsq_gemm_act(args(bsq)) == bsq.ERR_ARCH
    assert bsq.bsq_gemm_act_backward(args(bsq)) == bsq.ERR_ARCH
    assert bsq.bsq_expert_gemm_wgrad(bsq.MXFP8, P, P, P, P, P, P, 256, 128, 128, 2, P) == bsq.ERR_ARCH


def test_unknown_activations_and_dtypes_are_refused(bsq):
    q = bsq.QTensor(bsq.MXFP8, 4, 128, torch.zeros(512, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError, match="activation"):
        bsq.gemm_act(q, q, activation="tanh")
    with pytest.raises(ValueError, match="activation"):
        bsq.gemm_act_backward(q, q, activation="erf")
    with pytest.raises(TypeError):
        bsq.gemm_act(q, q, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        bsq.gemm_act(q, q, residual=torch.zeros(4, 4), out_dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="depth"):
        bsq.gemm_act(q, bsq.QTensor(bsq.MXFP8, 4, 256, q.codes, q.scales))
    c, o = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        bsq.expert_gemm(q, q, c.long(), o)
    with pytest.raises(AssertionError):
        bsq.expert_gemm(q, q, c, o)  # not on a GPU


def test_tensors_of_another_device_are_refused_before_any_launch(bsq, monkeypatch):
    class On(torch.Tensor):
        @property
        def is_cuda(self):
            return True

        def get_device(self):
            return self.gpu

    def on(t, gpu):
        t = t.as_subclass(On)
        t.gpu = gpu
        return t

    class Sizes:
        def __getattr__(self, name):
            if name in ("bsq_codes_bytes", "bsq_scales_bytes", "bsq_gemm_act_backward_workspace"):
                return lambda *a: 0
            raise AssertionError("the library was called: " + name)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bsq, "_fast", None)
    monkeypatch.setattr(bsq, "_lib", Sizes())
    monkeypatch.setattr(bsq, "_handle", lambda t: 0)
    u8 = dict(dtype=torch.uint8)
    bf = torch.zeros(4, 128, dtype=torch.bfloat16)
    parts = [torch.zeros(512, **u8)] * 4 + [torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)]

    def q(codes, scales):
        return bsq.QTensor(bsq.MXFP8, 4, 128, codes, scales)

    def forward(a, b, c, d, cnt, off, residual, out):
        bsq.gemm_act(q(a, b), bsq.QTensor(bsq.MXFP8, 128, 128, c, d), residual=residual, out=out)

    def backward(a, b, c, d, cnt, off, pre, out):
        bsq.expert_gemm_backward(q(a, b), bsq.QTensor(bsq.MXFP8, 128, 128, c, d), cnt, off, pre, "silu", out=out)

    def wgrad(a, b, c, d, cnt, off, _, out):
        bsq.expert_gemm_wgrad(q(a, b), bsq.QTensor(bsq.MXFP8, 128, 128, c, d), cnt, off, out=out)

    for call, skip, shape in ((forward, (4, 5), (4, 128)), (backward, (), (4, 128)), (wgrad, (6,), (1, 4, 128))):
        tensors = parts + [bf, bf.clone().reshape(shape)]
        for elsewhere in range(len(tensors)):
            if elsewhere not in skip:
                given = [on(t.clone(), 1 if i == elsewhere else 0) for i, t in enumerate(tensors)]
                with pytest.raises(AssertionError, match="current device"):
                    call(*given)
