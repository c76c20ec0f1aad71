"""How the functions around the linear layers hand a call on: streams, errors of the library, and
what a failed call leaves."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    return b


@pytest.mark.parametrize("fast", [True, False])
def test_a_stream_handle_of_zero_runs_behind_the_default_stream(bsq, monkeypatch, fast):
    """The inputs are written on the default stream after a wait of some 10 ms; a call with the default
    stream's handle comes after that, and its results are the default stream's."""
    if not fast:
        monkeypatch.setattr(bsq, "_fast", None)
    handle = torch.cuda.default_stream().cuda_stream
    assert handle == 0 and bsq._torch_stream(handle).cuda_stream == 0
    g = torch.Generator(device="cuda").manual_seed(1)
    new = torch.randn(64, 256, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(0, 8, (64, 2), device="cuda", generator=g)
    x, late_ids, w = torch.zeros_like(new), torch.zeros_like(ids), torch.full((64, 2), 0.5, device="cuda")
    grad = torch.zeros(64, 256, device="cuda")

    def calls(x, ids, grad, **kw):
        f = bsq.block_norm(x, x, **kw)
        r = bsq.block_norm_backward(x, x, f.x_out, x, f.stats, **kw)
        s = bsq.expert_sort(ids, 8, **kw)
        rows = bsq.expert_gather(x, s.position, s.slot, **kw)
        return (f.y, r.dx, *s, rows, bsq.expert_combine(rows, s.position, w, **kw),
                *bsq.expert_combine_backward(x, rows, s.position, s.slot, w, **kw),
                bsq.grad_norm([grad], **kw), bsq.clip_grad_norm([grad], 1.0, **kw), grad)

    want = calls(new, ids, new.float())
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    x.copy_(new)
    late_ids.copy_(ids)
    grad.copy_(new)
    got = calls(x, late_ids, grad, stream=handle)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert bsq.device_status() == 0


@pytest.fixture()
def fake_library(bsq):
    """The C++ host side with some of the library's functions replaced by Python ones."""
    import ctypes

    kept = []

    def install(**fakes):
        addresses = []
        for name in bsq._FAST_CALLS:
            f = getattr(bsq._lib, name)
            if name in fakes:
                f = ctypes.CFUNCTYPE(f.restype, *f.argtypes)(fakes[name])
                kept.append(f)
            addresses.append(ctypes.cast(f, ctypes.c_void_p).value)
        bsq._fast.init(*addresses)

    yield install
    install()


def test_clipping_whose_launch_fails_does_not_clip_again(bsq, fake_library):
    """The library scales all gradients in place and then reports a failed launch, as it may with more than
    1024 tensors: the call is not repeated by the Python code."""
    calls = []

    def clip(count, items, kind, max_norm, eps, norm, ws, nbytes, stream):
        calls.append(count)
        assert bsq._lib.bsq_clip_grad_norm(count, items, kind, max_norm, eps, norm, ws, nbytes, stream) == bsq.OK
        return bsq.ERR_LAUNCH

    fake_library(bsq_clip_grad_norm=clip)
    g = torch.full((100,), 4.0, device="cuda")
    with pytest.raises(bsq.BsqError) as e:
        bsq.clip_grad_norm([g], 4.0, eps=0.0)  # a norm of 40: the coefficient is 0.1, once
    assert e.value.code == bsq.ERR_LAUNCH and calls == [1]
    assert torch.allclose(g, torch.full_like(g, 0.4), rtol=1e-6, atol=0.0)


def test_refusals_of_the_library_leave_the_rest_to_the_python_code(bsq, fake_library):
    fake_library(bsq_block_norm=lambda args, stream: bsq.ERR_SHAPE)
    x = torch.randn(4, 64, device="cuda")
    y = bsq.block_norm(x, x).y
    fake_library()
    assert torch.equal(y, bsq.block_norm(x, x).y)


def test_every_failed_launch_is_raised(bsq, fake_library):
    fail = {n: (lambda *args: bsq.ERR_LAUNCH) for n in bsq._FAST_CALLS
            if not n.endswith("workspace") and not n.endswith("capacity")}
    x, w = torch.randn(4, 64, device="cuda"), torch.rand(4, 2, device="cuda")
    f = bsq.block_norm(x, x)
    s = bsq.expert_sort(torch.zeros(4, 2, device="cuda", dtype=torch.int64), 8)
    rows = bsq.expert_gather(x, s.position, s.slot)
    fake_library(**fail)
    for call in (lambda: bsq.block_norm(x, x), lambda: bsq.block_norm_backward(x, x, f.x_out, x, f.stats),
                 lambda: bsq.expert_sort(torch.zeros(4, 2, device="cuda", dtype=torch.int64), 8),
                 lambda: bsq.expert_gather(x, s.position, s.slot), lambda: bsq.expert_combine(rows, s.position, w),
                 lambda: bsq.expert_combine_backward(x, rows, s.position, s.slot, w), lambda: bsq.grad_norm([x]),
                 lambda: bsq.clip_grad_norm([x], 1.0)):
        with pytest.raises(bsq.BsqError) as e:
            call()
        assert e.value.code == bsq.ERR_LAUNCH
