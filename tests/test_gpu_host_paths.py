"""The C++ host side of the functions around the linear layers against the Python code of the same
functions: the same library calls, so the same bits, and the same refusals."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def bsq():
    import block_scaled_precision_bsq_gb300 as b

    assert b._fast is not None, "the C++ host side is not built"
    return b


def rand(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def both(bsq, monkeypatch, call):
    """The call through the C++ host side (which must take it) and through the Python code."""
    taken = []

    class Spy:
        def __getattr__(self, name):
            f = getattr(fast, name)

            def run(*args):
                r = f(*args)
                taken.append(r is not None)
                return r

            return run

    fast = bsq._fast
    monkeypatch.setattr(bsq, "_fast", Spy())
    a = call()
    assert taken and all(taken)
    monkeypatch.setattr(bsq, "_fast", None)
    b = call()
    monkeypatch.setattr(bsq, "_fast", fast)
    return a, b


def same(a, b):
    if a is None or b is None:
        assert a is None and b is None
    elif isinstance(a, torch.Tensor):
        assert a.dtype == b.dtype and a.shape == b.shape and a.is_contiguous() and torch.equal(a, b)
    else:
        assert type(a) is type(b) and len(a) == len(b)
        for x, y in zip(a, b):
            same(x, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
def test_block_norm(bsq, monkeypatch, dtype, groups, post, pre):
    h, x, d, dy = (rand(24, 200, dtype=dtype, seed=i) for i in range(4))
    wide = rand(24, 256, dtype=dtype, seed=9)
    w = [rand(200, dtype=torch.float32, seed=10 + i) for i in range(4)]
    gate = rand(groups, 200, dtype=torch.float32, seed=20) if groups > 1 else rand(200, dtype=torch.float32, seed=20)
    kw = dict(kind="layer", post_norm=post, post_weight=w[0] if post else None, post_bias=w[1] if post else None,
              gate=gate, residual_scale=0.5, weight_offset=1.0)
    prekw = dict(pre_weight=w[2], pre_bias=w[3]) if pre else {}
    for hh in (h, wide[:, 8:208]):
        f, g = both(bsq, monkeypatch, lambda: bsq.block_norm(hh, x, pre_norm=pre, **kw, **prekw))
        same(f, g)
        for grads in (True, False):
            same(*both(bsq, monkeypatch, lambda: bsq.block_norm_backward(d, dy if pre else None, f.x_out, hh, f.stats,
                                                                         param_grads=grads, **kw, **prekw)))
    same(*both(bsq, monkeypatch, lambda: bsq.block_norm(None, x, kind="rms")))
    empty = x[:0]
    same(*both(bsq, monkeypatch, lambda: bsq.block_norm(empty, empty, pre_norm=pre, **kw, **prekw)))


@pytest.mark.parametrize("tokens,topk,experts,align", [(0, 2, 4, 1), (1, 8, 64, 128), (500, 2, 16, 4), (20000, 4, 60, 1)])
def test_experts(bsq, monkeypatch, tokens, topk, experts, align):
    for dtype in (torch.int64, torch.int32):
        ids = torch.randint(-1, experts, (tokens, topk), device="cuda", dtype=dtype)
        s, t = both(bsq, monkeypatch, lambda: bsq.expert_sort(ids, experts, align=align))
        same(s, t)
    x, y = rand(tokens, 136), rand(s.slot.numel(), 136, seed=1)
    w = torch.rand(tokens, topk, device="cuda")
    same(*both(bsq, monkeypatch, lambda: bsq.expert_gather(x, s.position, s.slot)))
    same(*both(bsq, monkeypatch, lambda: bsq.expert_combine(y, s.position, w)))
    same(*both(bsq, monkeypatch, lambda: bsq.expert_gather_backward(y, s.position)))
    same(*both(bsq, monkeypatch, lambda: bsq.expert_combine_backward(x, y, s.position, s.slot, w)))


def test_gradient_norms(bsq, monkeypatch):
    ts = [rand(1 + 37 * i, dtype=torch.bfloat16 if i % 3 else torch.float32, seed=i) for i in range(150)]
    outs = [torch.zeros_like(t) for t in ts]
    for kind in (2.0, math.inf):
        same(*both(bsq, monkeypatch, lambda: bsq.grad_norm(ts, kind)))
        same(*both(bsq, monkeypatch, lambda: (bsq.clip_grad_norm(ts, 0.5, kind, outs=outs), *[o.clone() for o in outs])))
    same(*both(bsq, monkeypatch, lambda: (lambda c: (bsq.clip_grad_norm(c, 0.5), *c))([t.clone() for t in ts])))
    same(*both(bsq, monkeypatch, lambda: bsq.grad_norm(tuple(ts))))


def test_what_is_not_plain_is_refused_as_without_it(bsq):
    x, y = rand(8, 64), rand(8, 64, seed=1)
    w = rand(64)
    with pytest.raises(TypeError):
        bsq.block_norm(x, y.float())
    with pytest.raises(TypeError):
        bsq.block_norm(x, y, pre_weight=w, gate=w.float())
    with pytest.raises(AssertionError):
        bsq.block_norm(x, y[:4])
    with pytest.raises(AssertionError):
        bsq.block_norm(x, y, pre_weight=w[:32])
    with pytest.raises(AssertionError):
        bsq.block_norm(x.t(), y.t())
    with pytest.raises(AssertionError):
        bsq.block_norm(x, y, pre_norm=False, pre_weight=w)
    with pytest.raises(KeyError):
        bsq.block_norm(x, y, kind="batch")
    with pytest.raises(bsq.BsqError):
        bsq.block_norm(x, y, eps=-1.0)
    with pytest.raises(bsq.BsqError):
        bsq.block_norm(x, y, gate=rand(3, 64))  # 8 rows, 3 gates
    f = bsq.block_norm(x, y)
    with pytest.raises(AssertionError):
        bsq.block_norm_backward(None, x, f.x_out, y, f.stats[:4])
    with pytest.raises(AssertionError):
        bsq.block_norm_backward(None, x, None, y, f.stats)
    with pytest.raises(TypeError):
        bsq.expert_sort(torch.zeros(4, 2, device="cuda"), 8)
    with pytest.raises(bsq.BsqError):
        bsq.expert_sort(torch.zeros(4, 2, device="cuda", dtype=torch.int64), 0)
    with pytest.raises(bsq.BsqError):
        bsq.expert_sort(torch.zeros(4, 2, device="cuda", dtype=torch.int64), 4096)
    s = bsq.expert_sort(torch.zeros(8, 2, device="cuda", dtype=torch.int64), 4)
    with pytest.raises(TypeError):
        bsq.expert_gather(x, s.position.long(), s.slot)
    with pytest.raises(AssertionError):
        bsq.expert_gather(x[:4], s.position, s.slot)
    with pytest.raises(TypeError):
        bsq.expert_combine(rand(16, 64), s.position, rand(8, 2))
    with pytest.raises(AssertionError):
        bsq.expert_combine_backward(x, rand(15, 64), s.position, s.slot, torch.rand(8, 2, device="cuda"))
    with pytest.raises(TypeError):
        bsq.clip_grad_norm([x.half()], 1.0)
    with pytest.raises(AssertionError):
        bsq.clip_grad_norm([x.t()], 1.0)
    with pytest.raises(AssertionError):
        bsq.clip_grad_norm([x], 1.0, outs=[y[:4]])
    with pytest.raises(bsq.BsqError):
        bsq.clip_grad_norm([x], -1.0)
    assert bsq.device_status() == 0
