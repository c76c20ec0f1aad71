"""Refusals of the block norms, expert rows and gradient norms that need no GPU: every invalid
argument is turned away before any CUDA call."""
import ctypes

import pytest
import torch

P = 1 << 20  # a 16-byte aligned dummy address: never dereferenced on these paths


@pytest.fixture(scope="module")
def bsq():
    import __graft_entry__

    __graft_entry__.build()
    import block_scaled_precision_bsq_gb300 as b

    return b


def _norm(bsq, **kw):
    a = dict(kind=2, flags=0, rows=4, cols=64, gate_groups=1, eps=1e-6, residual_scale=1.0, weight_offset=0.0, h=P, x=P,
             h_stride=64, x_stride=64, x_out=P, y=P, stats=P)
    a.update(kw)
    return bsq.bsq_block_norm(bsq.BlockNormArgs(**a), None)


def test_block_norm_refusals(bsq):
    nan, inf = float("nan"), float("inf")
    assert bsq._lib.bsq_block_norm(None, None) == bsq.ERR_ARG
    for bad in (dict(kind=0), dict(kind=3), dict(flags=0x4000), dict(rows=-1), dict(cols=0), dict(gate_groups=0),
                dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(residual_scale=nan), dict(weight_offset=inf),
                dict(x=None), dict(x_out=None, y=None), dict(h=None, gate=P),
                dict(h=None, flags=bsq.FLAG_POST_NORM)):
        assert _norm(bsq, **bad) == bsq.ERR_ARG, bad
    for bad in (dict(rows=1 << 31), dict(cols=65537), dict(cols=32769, flags=bsq.FLAG_SRC_F32),
                dict(gate_groups=3, gate=P), dict(h_stride=-1), dict(x_stride=1 << 31)):
        assert _norm(bsq, **bad) == bsq.ERR_SHAPE, bad
    for bad in (dict(h=P + 1), dict(x=P + 2, flags=bsq.FLAG_SRC_F32), dict(y=P + 1), dict(x_out=P + 1),
                dict(pre_weight=P + 1), dict(gate=P + 2, flags=bsq.FLAG_PARAMS_F32), dict(stats=P + 4)):
        assert _norm(bsq, **bad) == bsq.ERR_ALIGN, bad


def _grad(bsq, **kw):
    a = dict(kind=2, flags=bsq.FLAG_POST_NORM, rows=4, cols=64, gate_groups=1, residual_scale=1.0, weight_offset=0.0,
             dx_out=P, dy=P, x_out=P, h=P, dx_out_stride=64, dy_stride=64, x_out_stride=64, h_stride=64, stats=P, dx=P,
             dh=P)
    a.update(kw)
    return bsq.bsq_block_norm_backward(bsq.BlockNormGradArgs(**a), None)


def test_block_norm_backward_refusals(bsq):
    assert bsq._lib.bsq_block_norm_backward(None, None) == bsq.ERR_ARG
    for bad in (dict(kind=0), dict(flags=0x4000), dict(rows=-1), dict(cols=-5), dict(dx_out=None, dy=None),
                dict(x_out=None), dict(stats=None), dict(h=None), dict(flags=0, dpost_weight=P),
                dict(flags=0, dpost_bias=P), dict(dpre_weight=P), dict(dgate=P, h=None, flags=0, workspace=P)):
        assert _grad(bsq, **bad) == bsq.ERR_ARG, bad
    for bad in (dict(rows=1 << 31), dict(cols=65537), dict(gate_groups=3), dict(dy_stride=-1)):
        assert _grad(bsq, **bad) == bsq.ERR_SHAPE, bad
    for bad in (dict(dy=P + 1), dict(dx=P + 1), dict(stats=P + 8), dict(dpre_bias=P + 2, workspace=P),
                dict(dpre_bias=P, workspace=P + 8)):
        assert _grad(bsq, **bad) == bsq.ERR_ALIGN, bad
    ws = bsq.bsq_block_norm_backward_workspace
    assert ws(0, -1, 64) == 0 and ws(0, 4, 0) == 0 and ws(0, 4, 64, 3) == 0 and ws(0x4000, 4, 64) == 0


def test_expert_capacity(bsq):
    cap = bsq.bsq_expert_capacity
    assert cap(0, 8, 128) == 0
    assert cap(1, 8, 1) == 1
    assert cap(1, 8, 128) == 128       # one slot fills one expert's segment
    assert cap(100, 8, 1) == 100
    assert cap(100, 2, 16) == 144      # 100 + 2 * 15 = 130, rounded up
    assert cap(-1, 8, 1) == 0 and cap(5, 0, 1) == 0 and cap(5, 8, 0) == 0 and cap(5, 2049, 1) == 0
    # never less than any split of the slots needs
    for slots in (1, 5, 31, 64):
        for experts in (1, 3, 8):
            for align in (1, 4, 16):
                worst = max(sum(-(-c // align) * align for c in split)
                            for split in ([slots] + [0] * (experts - 1),
                                          [slots // experts + (i < slots % experts) for i in range(experts)],
                                          [1] * min(experts - 1, slots - 1) + [slots - min(experts - 1, slots - 1)]))
                assert cap(slots, experts, align) >= worst


def test_expert_refusals(bsq):
    E, S, A = bsq.ERR_ARG, bsq.ERR_SHAPE, bsq.ERR_ALIGN
    so = bsq.bsq_expert_sort
    assert so(0x100, P, 4, 2, 8, 1, 8, P, P, P, P) == E           # flag
    assert so(0, P, -1, 2, 8, 1, 8, P, P, P, P) == E
    assert so(0, P, 4, 0, 8, 1, 8, P, P, P, P) == E
    assert so(0, P, 4, 2, 0, 1, 8, P, P, P, P) == E
    assert so(0, P, 4, 2, 8, 0, 8, P, P, P, P) == E
    assert so(0, None, 4, 2, 8, 1, 8, P, P, P, P) == E
    assert so(0, P, 4, 2, 8, 1, 8, None, P, P, P) == E
    assert so(0, P, 4, 2, 8, 1, 8, P, P, P, None) == E
    assert so(0, P, 4, 2, 8, 1, 7, P, P, P, P) == S               # capacity too small
    assert so(0, P, 4, 2, 2049, 1, 8, P, P, P, P) == S            # experts
    assert so(0, P, 1 << 30, 2, 8, 1, 1 << 30, P, P, P, P) == S   # 2^31 slots
    assert so(bsq.FLAG_IDS_I64, P + 4, 4, 2, 8, 1, 8, P, P, P, P) == A
    assert so(0, P, 4, 2, 8, 1, 8, P, P + 2, P, P) == A
    many = 65536
    assert bsq.bsq_expert_sort_workspace(many * 2, 8) > 0 and bsq.bsq_expert_sort_workspace(8, 8) == 0
    assert so(0, P, many, 2, 8, 1, many * 2, P, P, P, P) == E     # no workspace
    assert so(0, P, many, 2, 8, 1, many * 2, P, P, P, P, P, bsq.bsq_expert_sort_workspace(many * 2, 8) - 1) == E
    g = bsq.bsq_expert_gather
    assert g(0x200, P, 64, P, P, 4, 2, 64, 8, P) == E
    assert g(0, None, 64, P, P, 4, 2, 64, 8, P) == E
    assert g(0, P, 64, None, P, 4, 2, 64, 8, P) == E
    assert g(0, P, 64, P, None, 4, 2, 64, 8, P) == E
    assert g(0, P, 64, P, P, 4, 2, 0, 8, P) == E
    assert g(0, P, -1, P, P, 4, 2, 64, 8, P) == S
    assert g(0, P + 1, 64, P, P, 4, 2, 64, 8, P) == A
    c = bsq.bsq_expert_combine
    assert c(0, P, 64, None, P, 4, 2, 64, 8, P) == E
    assert c(0, None, 64, P, P, 4, 2, 64, 8, P) == E
    assert c(0, P, 64, P, P, 4, 2, 64, 8, None) == E
    assert c(0, P, 64, P, P, 4, 2, 64, 1 << 31, P) == S
    assert c(0, P, 64, P, P + 2, 4, 2, 64, 8, P) == A
    b = bsq.bsq_expert_combine_backward
    assert b(0, None, 64, P, 64, P, P, P, 4, 2, 64, 8, P, P) == E
    assert b(0, P, 64, P, 64, P, P, None, 4, 2, 64, 8, P, P) == E
    assert b(0, P, 64, P, 64, P, P, P, 4, 2, 64, 8, None, P) == E
    assert b(0, P, 64, P, 64, P, P, P, 4, 2, 64, 8, P, None) == E
    assert b(0, P, 64, P, -64, P, P, P, 4, 2, 64, 8, P, P) == S
    assert b(bsq.FLAG_SRC_F32, P, 64, P + 2, 64, P, P, P, 4, 2, 64, 8, P, P) == A


def test_grad_norm_refusals(bsq):
    E, S, A = bsq.ERR_ARG, bsq.ERR_SHAPE, bsq.ERR_ALIGN
    ok = [(P, P, 10, True)]
    clip = bsq.bsq_clip_grad_norm
    assert bsq._lib.bsq_grad_norm(-1, None, 1, P, P, 1 << 20, None) == E
    assert bsq._lib.bsq_grad_norm(1, None, 1, P, P, 1 << 20, None) == E
    assert bsq.bsq_grad_norm(ok, 3, P, P, 1 << 20) == E
    assert bsq.bsq_grad_norm(ok, 1, None, P, 1 << 20) == E
    assert bsq.bsq_grad_norm(ok, 1, P, None, 1 << 20) == E
    assert bsq.bsq_grad_norm([(None, None, 10, True)], 1, P, P, 1 << 20) == E
    assert bsq.bsq_grad_norm([(P, None, -1, True)], 1, P, P, 1 << 20) == E
    assert bsq.bsq_grad_norm([(P, None, 1 << 41, True)], 1, P, P, 1 << 20) == S
    assert bsq.bsq_grad_norm([(P + 2, None, 4, True)], 1, P, P, 1 << 20) == A
    assert bsq.bsq_grad_norm(ok, 1, P + 2, P, 1 << 20) == A
    assert bsq.bsq_grad_norm(ok, 1, P, P + 8, 1 << 20) == A
    assert clip([(P, None, 10, True)], 1, 1.0, 0.0, P, P, 1 << 20) == E   # no destination
    assert clip(ok, 1, -1.0, 0.0, P, P, 1 << 20) == E
    assert clip(ok, 1, float("nan"), 0.0, P, P, 1 << 20) == E
    assert clip(ok, 1, 1.0, -1.0, P, P, 1 << 20) == E
    assert clip(ok, 1, 1.0, float("inf"), P, P, 1 << 20) == E
    assert clip([(P, P + 1, 4, False)], 1, 1.0, 0.0, P, P, 1 << 20) == A
    assert bsq.bsq_clip_grad_norm_workspace(-1) == 0
    with pytest.raises(ValueError):
        bsq._norm_kind(1.0)


def test_python_layer_refuses_cpu_tensors_and_wrong_types(bsq):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError):
        bsq.block_norm(x, x)
    with pytest.raises(TypeError):
        bsq.block_norm(None, x.half())
    with pytest.raises(TypeError):
        bsq.expert_sort(torch.zeros(4, 2), 8)
    with pytest.raises(AssertionError):
        bsq.expert_sort(torch.zeros(4, 2, dtype=torch.int64), 8)
    with pytest.raises(TypeError):
        bsq.clip_grad_norm([x.half()], 1.0)
    with pytest.raises(AssertionError):
        bsq.clip_grad_norm([x], 1.0, outs=[])
    assert ctypes.sizeof(bsq.GradItem) == 32
