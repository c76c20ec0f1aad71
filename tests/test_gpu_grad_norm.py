"""grad_norm and clip_grad_norm against 64-bit sums.

A thread adds at most 64 squares in fp32 before it goes to fp64, so the sum of squares is off by at
most 65 u of itself (u = 2^-24) and the norm by half of that, rounded to fp32 once more."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TOL = 33 * U + 2 * U


def _bsq():
    import block_scaled_precision_bsq_gb300 as bsq

    return bsq


def exact_norm(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def check(tensors, max_norm=1.0, eps=1e-6, outs=None):
    bsq = _bsq()
    want = exact_norm(tensors)
    got = bsq.grad_norm(tensors)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(float(got) - want) <= TOL * want, (float(got), want)
    big = max([float(t.abs().max()) for t in tensors if t.numel()] or [0.0])
    assert float(bsq.grad_norm(tensors, norm_type=math.inf)) == big
    ref = [t.double() for t in tensors]
    n = bsq.clip_grad_norm(tensors, max_norm, eps=eps, outs=outs)
    assert torch.equal(n, got)
    coef = min(1.0, max_norm / (want + eps))
    for o, r in zip(outs if outs is not None else tensors, ref):
        # the coefficient carries the norm's error, a sum and a quotient; then one product and one rounding
        hs = torch.finfo(o.dtype).eps / 2
        e = (TOL + 4 * U) * (r * coef).abs()
        tiny = torch.finfo(torch.float32).tiny  # below the normal range a step is 2^-133 (bf16) or less
        assert ((o.double() - r * coef).abs() <= e + hs * ((r * coef).abs() + e) + (tiny * hs if coef < 1 else 0)).all()
    return float(n)


def rand(n, std=1.0, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + n)
    return (torch.randn(n, device="cuda", generator=g) * std).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [[1], [0], [7], [0, 5, 0, 0, 3, 0], [16384], [16383], [16385], [100000, 3, 12345],
                                   [1 << 22, 17]])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
def test_sizes(sizes, dtype, max_norm):
    check([rand(n, 0.1, dtype) for n in sizes], max_norm)


def test_mixed_types_many_tensors():
    ts = [rand(1 + (i * 37) % 501, 0.01, torch.bfloat16 if i % 3 else torch.float32, i) for i in range(2600)]
    check(ts, 0.3)
    check(ts[:64], 0.3)
    check(ts[:65], 0.3)
    check(ts[:1025], 0.3)


def test_no_tensors():
    bsq = _bsq()
    assert float(bsq.grad_norm([])) == 0.0
    assert float(bsq.clip_grad_norm([], 1.0)) == 0.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_odd_addresses_and_other_destinations(dtype):
    base = rand(40000, 0.1, dtype)
    for shift in (1, 2, 3, 5):
        ts = [base[shift:20001], base[20003 + shift:39990]]
        for to in (0, 1, shift):
            room = torch.full((40010,), 7.0, dtype=dtype, device="cuda")
            outs, at = [], to
            for t in ts:
                outs.append(room[at:at + t.numel()])
                at += t.numel() + 3
            keep = base.clone()
            check(ts, 0.25, outs=outs)
            assert torch.equal(base, keep)                       # the sources stay
            assert (room[:to] == 7).all() and (room[at - 3:] == 7).all()  # nothing around the outputs is written
            assert (room[to + ts[0].numel():to + ts[0].numel() + 3] == 7).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-12, 1e12, 1e19, 1e30])
def test_whole_range_of_fp32(scale):
    """Squares of these would lose bits or overflow in fp32."""
    check([rand(50001, scale), rand(3, scale)], max_norm=scale)


def test_one_large_and_many_tiny_values():
    t = rand(70000, 1e-25)
    t[40000] = 1e-3
    check([t])
    check([rand(100000, 1e-25), rand(100000, 1e20)])


def test_nothing_to_clip_leaves_every_bit():
    bsq = _bsq()
    t = rand(30000, 1e-4)
    keep = t.clone()
    bsq.clip_grad_norm([t], 100.0)
    assert torch.equal(t, keep)
    o = torch.empty_like(t)
    bsq.clip_grad_norm([t], 100.0, outs=[o])
    assert torch.equal(o, keep)
    bsq.clip_grad_norm([t], math.inf)
    assert torch.equal(t, keep)


def test_nan_and_infinity():
    bsq = _bsq()
    for bad, other in ((math.nan, math.inf), (math.inf, 1.0), (-math.inf, 1.0)):
        a, b = rand(20000), rand(99, 1.0, torch.bfloat16)
        a[12345] = bad
        b[7] = other
        n, m = float(bsq.grad_norm([a, b])), float(bsq.grad_norm([a, b], norm_type=math.inf))
        if math.isnan(bad):
            assert math.isnan(n) and math.isnan(m)
            bsq.clip_grad_norm([a, b], 1.0)
            assert a.isnan().all() and b.isnan().all()
        else:
            assert n == math.inf and m == math.inf
            bsq.clip_grad_norm([a, b], 1.0)  # coefficient 0: finite values become 0, infinities NaN
            assert a[12345].isnan() and (a[:12345] == 0).all() and (b == 0).all()


def test_max_norm_clipping():
    bsq = _bsq()
    a, b = rand(20000), rand(501, 3.0, torch.bfloat16)
    big = max(float(a.abs().max()), float(b.abs().max()))
    ra, rb = a.double(), b.double()
    assert float(bsq.clip_grad_norm([a, b], 0.5, norm_type=math.inf, eps=0.0)) == big
    assert ((a.double() - ra * (0.5 / big)).abs() <= 3 * U * a.double().abs() + 1e-30).all()
    assert ((b.double() - rb * (0.5 / big)).abs() <= 2.0 ** -8 * (1 + 2.0 ** -8) * (rb * (0.5 / big)).abs() + 1e-30).all()


def test_same_bits_on_another_stream_and_in_a_graph():
    bsq = _bsq()
    ts = [rand(1 + i * 997, 0.1, torch.bfloat16 if i % 2 else torch.float32, i) for i in range(100)]
    outs = [[torch.empty_like(t) for t in ts] for _ in range(3)]
    n0 = bsq.clip_grad_norm(ts, 0.5, outs=outs[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    n1 = bsq.clip_grad_norm(ts, 0.5, outs=outs[1], stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n2 = bsq.clip_grad_norm(ts, 0.5, outs=outs[2])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n0, n1) and torch.equal(n0, n2)
    for a, b, c in zip(*outs):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_more_than_2_31_elements():
    n = (1 << 31) + 12345
    t = torch.empty(n, dtype=torch.bfloat16, device="cuda").fill_(2.0 ** -10)
    t[-1] = 3.0
    bsq = _bsq()
    want = math.sqrt((n - 1) * 2.0 ** -20 + 9.0)
    got = float(bsq.clip_grad_norm([t], 1.0))
    assert abs(got - want) <= TOL * want
    coef = torch.tensor(1.0) / (torch.tensor(got) + 1e-6)
    for i in (0, (1 << 31) - 1, 1 << 31, n - 2):
        assert float(t[i]) == float((2.0 ** -10 * coef).to(torch.bfloat16))
    assert float(t[-1]) == float((3.0 * coef).to(torch.bfloat16))


def test_small_workspace_is_refused():
    bsq = _bsq()
    t, norm = rand(100), torch.empty((), device="cuda")
    n = bsq.bsq_clip_grad_norm_workspace(1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    items = [(t, t, 100, True)]
    assert bsq.bsq_grad_norm(items, 1, norm, ws, n - 1) == bsq.ERR_ARG
    assert bsq.bsq_clip_grad_norm(items, 1, 1.0, 0.0, norm, ws, n - 1) == bsq.ERR_ARG
    assert bsq.bsq_grad_norm(items, 1, norm, ws, n) == bsq.OK
    assert bsq.device_status() == 0
