"""How the functions around the linear layers hand a call on, without a GPU: streams, devices and the
C++ host side are stood in for."""
import pytest
import torch


@pytest.fixture(scope="module")
def bsq():
    import __graft_entry__

    __graft_entry__.build()
    import block_scaled_precision_bsq_gb300 as b

    return b


def test_a_stream_handle_of_zero_is_the_default_stream(bsq, monkeypatch):
    """torch.cuda.default_stream().cuda_stream is 0, and 0 is the library's legacy default stream too."""
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    assert bsq._torch_stream(0) == "default"
    assert bsq._torch_stream(1 << 40) == ("external", 1 << 40)


class OnGpu(torch.Tensor):
    """A CPU tensor that says that it lies on a GPU (`gpu`), for checks that come before any launch."""

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        name = getattr(func, "__name__", "")
        if func == torch.Tensor.is_cuda.__get__:
            return True
        if name == "get_device":
            return args[0].gpu
        r = super().__torch_function__(func, types, args, kwargs or {})
        if isinstance(r, OnGpu) and not hasattr(r, "gpu"):
            r.gpu = args[0].gpu
        return r


def on_gpu(t, gpu):
    t = t.as_subclass(OnGpu)
    t.gpu = gpu
    return t


class NoCalls:
    """In the place of the library: any call would be a launch."""

    def __getattr__(self, name):
        raise AssertionError("the library was called: " + name)


@pytest.fixture()
def gpu_zero(bsq, monkeypatch):
    """GPU 0 is current, nothing may be allocated on a GPU or launched."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bsq, "_fast", None)
    monkeypatch.setattr(bsq, "_lib", NoCalls())
    monkeypatch.setattr(bsq, "_handle", lambda t: 0)
    return bsq


def test_tensors_of_another_device_are_refused_before_any_launch(gpu_zero):
    """All on GPU 1 while GPU 0 is current, or one of them: a launch would run on GPU 0 with GPU 1's addresses."""
    bsq = gpu_zero
    m = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, pos, slot = torch.zeros(64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    ids, weights, y = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2), torch.zeros(8, 64, dtype=torch.bfloat16)
    stats, v = torch.zeros(4, 4), torch.zeros(10)
    kw = dict(kind="layer", post_norm=True)

    def norm(h, x, pw, pb, g, w2, b2):
        bsq.block_norm(h, x, post_weight=pw, post_bias=pb, gate=g, pre_weight=w2, pre_bias=b2, **kw)

    def norm_out(x, x_out, yy, st):
        bsq.block_norm(x, x, out=bsq.BlockNorm(x_out, yy, st))

    def norm_backward(dxo, dy, xo, h, st, pw, pb, g, w2, b2):
        bsq.block_norm_backward(dxo, dy, xo, h, st, post_weight=pw, post_bias=pb, gate=g, pre_weight=w2, pre_bias=b2, **kw)

    calls = [(norm, [m, m, w, w, w, w, w]), (norm_out, [m, m, m, stats]),
             (norm_backward, [m, m, m, m, stats, w, w, w, w, w]),
             (lambda i: bsq.expert_sort(i, 8), [ids]),
             (bsq.expert_gather, [m, pos, slot]), (lambda a, b, c, d: bsq.expert_gather(a, b, c, out=d), [m, pos, slot, y]),
             (bsq.expert_combine, [y, pos, weights]),
             (lambda a, b, c, d: bsq.expert_combine(a, b, c, out=d), [y, pos, weights, m]),
             (bsq.expert_combine_backward, [m, y, pos, slot, weights]),
             (lambda a, b: bsq.grad_norm([a, b]), [v, v]),
             (lambda a, b, c, d: bsq.clip_grad_norm([a, b], 1.0, outs=[c, d]), [v, v, v, v])]
    for call, tensors in calls:
        n = len(tensors)
        for elsewhere in [range(n)] + [[i] for i in range(n)]:
            args = [on_gpu(t.clone(), 1 if i in elsewhere else 0) for i, t in enumerate(tensors)]
            with pytest.raises(AssertionError, match="current device"):
                call(*args)


def test_a_failed_launch_is_raised_and_not_repeated(bsq, monkeypatch):
    """The C++ host side returns the code of a launch that failed; launches before it may have run (clipping
    in place), so the Python code must not call the library again."""

    class Failing:
        def __getattr__(self, name):
            return lambda *args: bsq.ERR_LAUNCH

    monkeypatch.setattr(bsq, "_fast", Failing())
    monkeypatch.setattr(bsq, "_lib", NoCalls())
    m, v, i = torch.zeros(4, 64), torch.zeros(8), torch.zeros(4, 2, dtype=torch.int32)
    for call, what in ((lambda: bsq.clip_grad_norm([v], 1.0), "bsq_clip_grad_norm"),
                       (lambda: bsq.grad_norm([v]), "bsq_grad_norm"), (lambda: bsq.block_norm(m, m), "bsq_block_norm"),
                       (lambda: bsq.block_norm_backward(m, m, m, m, v), "bsq_block_norm_backward"),
                       (lambda: bsq.expert_sort(i, 8), "bsq_expert_sort"),
                       (lambda: bsq.expert_gather(m, i, i), "bsq_expert_gather"),
                       (lambda: bsq.expert_combine(m, i), "bsq_expert_combine"),
                       (lambda: bsq.expert_combine_backward(m, m, i, i, v), "bsq_expert_combine_backward")):
        monkeypatch.setattr(bsq, "bsq_strerror", lambda code: "launch")
        with pytest.raises(bsq.BsqError, match=what) as e:
            call()
        assert e.value.code == bsq.ERR_LAUNCH


def _binding(bsq, monkeypatch, tmp_path, stamp):
    monkeypatch.setattr(bsq, "_HERE", str(tmp_path))
    (tmp_path / "_bsq_torch.so").write_bytes(b"not a module of this Python")
    if stamp is not None:
        (tmp_path / "_bsq_torch.so.torch").write_text(stamp)


def test_a_host_side_that_does_not_load_leaves_the_python_code(bsq, monkeypatch, tmp_path):
    """Whatever is wrong with the module, the package imports: the Python code of the same functions serves."""
    _binding(bsq, monkeypatch, tmp_path, bsq._binding_stamp())
    with pytest.warns(RuntimeWarning, match="_bsq_torch"):
        assert bsq._load_fast() is None


def test_a_host_side_of_another_torch_or_python_is_not_loaded(bsq, monkeypatch, tmp_path):
    import warnings

    this = bsq._binding_stamp()
    assert torch.__version__ in this
    for stamp in (None, "", torch.__version__, this.replace(torch.__version__, "0.0.0"), this + "x"):
        _binding(bsq, monkeypatch, tmp_path, stamp)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            assert bsq._load_fast() is None
        (tmp_path / "_bsq_torch.so.torch").unlink(missing_ok=True)


def test_the_built_host_side_is_loaded(bsq):
    assert bsq._load_fast() is not None and bsq._fast is not None


def test_expert_sort_refuses_sizes_before_it_allocates(bsq, monkeypatch):
    """2048 experts' segments of 2^21 rows would be a slot array of 17 GB, allocated only to be refused."""
    lib = bsq._lib
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bsq, "_fast", None)

    class Sizes(NoCalls):
        bsq_expert_capacity = staticmethod(lib.bsq_expert_capacity)
        bsq_strerror = staticmethod(lib.bsq_strerror)

    def no_allocation(*args, **kw):
        raise AssertionError("allocated")

    ids = on_gpu(torch.zeros(2048, 2, dtype=torch.int64), 0)
    none = on_gpu(torch.zeros(4, 0, dtype=torch.int64), 0)
    monkeypatch.setattr(torch, "empty", no_allocation)
    monkeypatch.setattr(bsq, "_lib", Sizes())
    for args, code in (((ids, 2048, 1 << 21), bsq.ERR_SHAPE), ((ids, 2049, 1), bsq.ERR_SHAPE),
                       ((ids, 8, 1 << 31), bsq.ERR_SHAPE), ((ids, 0, 1), bsq.ERR_ARG), ((ids, -3, 1), bsq.ERR_ARG),
                       ((ids, 8, 0), bsq.ERR_ARG), ((none, 8, 1), bsq.ERR_ARG)):
        with pytest.raises(bsq.BsqError) as e:
            bsq.expert_sort(*args)
        assert e.value.code == code, args[1:]


def test_linear_layers_refuse_tensors_of_another_device(gpu_zero, monkeypatch):
    bsq = gpu_zero
    monkeypatch.setattr(bsq, "bsq_gemm_splitk_splits", lambda *args: 2)
    x, w, b = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16), torch.zeros(1)
    out, ws = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(8192)

    def q(codes, scales, g=None):
        return bsq.QTensor(bsq.NVFP4 if g is not None else bsq.MXFP8, 64, 64, codes, scales, g)

    c, s = torch.zeros(4096, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    calls = [(lambda x, c, s: bsq.quantize("mxfp8", x, out=q(c, s)), [x, c, s]),
             (lambda x, c, s, g: bsq.quantize("nvfp4", x, global_scale=g, out=q(c, s, g)), [x, c, s, b]),
             (lambda x, y, c, s, d, t: bsq.quantize_many("mxfp8", [x, y], outs=[q(c, s), q(d, t)]), [x, x, c, s, c, s]),
             (lambda x, g, b, c, s: bsq.layernorm_quantize("mxfp8", x, g, b, out=q(c, s)), [x, w, w, c, s]),
             (lambda x, c, s, d, t: bsq.quantize_dual("mxfp8", x, out=(q(c, s), q(d, t))), [x, c, s, c, s]),
             (lambda c, s, g, o: bsq.delayed_global_scale(q(c, s, g), out=o), [c, s, b, b]),
             (lambda c, s, d, t, b, o: bsq.gemm(q(c, s), q(d, t), b, out=o), [c, s, c, s, w, out]),
             (lambda c, s, d, t, b, v, o: bsq.gemm_splitk(q(c, s), q(d, t), b, workspace=v, out=o), [c, s, c, s, w, ws, out]),
             (lambda c, s, d, t, b, o: bsq.gemm_gelu(q(c, s), q(d, t), b, out=o), [c, s, c, s, w, out]),
             (lambda c, s, d, t, b, e, u: bsq.gemm_gelu_quantize(q(c, s), q(d, t), b, out=q(e, u)), [c, s, c, s, w, c, s]),
             (lambda c, s, d, t, o: bsq.convt2x2(q(c, s), q(d, t), 1, 8, 8, out=o), [c, s, c, s, out])]
    for k, (call, tensors) in enumerate(calls):
        n = len(tensors)
        for elsewhere in [range(n)] + [[i] for i in range(n)]:
            args = [on_gpu(t.clone(), 1 if i in elsewhere else 0) for i, t in enumerate(tensors)]
            with pytest.raises(AssertionError, match="current device"):
                call(*args)
        with pytest.raises(AssertionError, match="the library was called"):  # all of them here: taken
            call(*[on_gpu(t.clone(), 0) for t in tensors])
