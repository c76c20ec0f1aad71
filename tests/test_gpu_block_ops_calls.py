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
