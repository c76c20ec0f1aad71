"""expert_sort, expert_gather, expert_combine and their gradients against plain loops and 64-bit sums."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F64 = torch.float64


def _bsq():
    import block_scaled_precision_bsq_gb300 as bsq

    return bsq


def plain_sort(ids, experts, align, capacity):
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(i)
    slot, offsets, position = [], [0], [-1] * len(flat)
    for members in lists:
        for i in members:
            position[i] = len(slot)
            slot.append(i)
        slot += [-1] * (-len(slot) % align)
        offsets.append(len(slot))
    assert len(slot) <= capacity
    slot += [-1] * (capacity - len(slot))
    i32 = dict(dtype=torch.int32)
    return (torch.tensor([len(m) for m in lists], **i32), torch.tensor(offsets, **i32),
            torch.tensor(position, **i32).reshape(ids.shape), torch.tensor(slot, **i32))


def make_ids(tokens, topk, experts, seed, kind="spread", dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":        # everything to one expert
        ids = torch.full((tokens, topk), experts - 1)
    elif kind == "none":     # every choice dropped
        ids = torch.full((tokens, topk), -1)
    elif kind == "outside":  # ids on both sides of the range, and far out of it
        ids = torch.randint(-3, experts + 3, (tokens, topk), generator=g)
        if ids.numel():
            ids.view(-1)[0] = torch.iinfo(dtype).max
            ids.view(-1)[-1] = torch.iinfo(dtype).min
    else:
        ids = torch.randint(0, experts, (tokens, topk), generator=g)
    return ids.to(dtype)


@pytest.mark.parametrize("tokens,topk,experts,align", [
    (0, 2, 8, 1), (0, 2, 8, 128), (1, 1, 1, 1), (1, 8, 64, 1), (1, 8, 64, 128), (5, 3, 7, 16), (31, 1, 2, 1), (33, 2, 1, 4),
    (256, 8, 256, 1), (255, 8, 257, 3), (1024, 2, 2048, 1), (1025, 2, 2048, 2), (4099, 4, 60, 128), (30011, 6, 128, 1),
    (100000, 8, 16, 128)])
@pytest.mark.parametrize("kind", ["spread", "one", "none", "outside"])
def test_sort(tokens, topk, experts, align, kind):
    bsq = _bsq()
    for dtype in (torch.int64, torch.int32):
        ids = make_ids(tokens, topk, experts, tokens + topk, kind, dtype)
        got = bsq.expert_sort(ids.cuda(), experts, align=align)
        assert got.slot.numel() == bsq.bsq_expert_capacity(tokens * topk, experts, align)
        want = plain_sort(ids, experts, align, got.slot.numel())
        for g, w, name in zip(got, want, got._fields):
            assert torch.equal(g.cpu(), w), name


def make_rows(tokens, topk, experts, cols, dtype, align=1, seed=0, kind="outside"):
    bsq = _bsq()
    ids = make_ids(tokens, topk, experts, seed, kind).cuda()
    s = bsq.expert_sort(ids, experts, align=align)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(tokens, cols, device="cuda", generator=g).to(dtype)
    y = torch.randn(s.slot.numel(), cols, device="cuda", generator=g).to(dtype)
    w = torch.rand(tokens, topk, device="cuda", generator=g)
    return s, x, y, w


def check_rows(s, x, y, w):
    bsq = _bsq()
    topk, hs = w.shape[1], torch.finfo(x.dtype).eps / 2
    rows = bsq.expert_gather(x, s.position, s.slot)
    live = s.slot >= 0
    want = torch.zeros_like(rows)
    want[live] = x[(s.slot[live] // topk).long()]
    assert torch.equal(rows, want)

    ok = (s.position >= 0)[..., None]
    picked = torch.where(ok, y.to(F64)[s.position.clamp(min=0).long()], 0.0) if y.shape[0] else \
        torch.zeros(*w.shape, y.shape[1], device="cuda", dtype=F64)
    for weights in (w, None):
        terms = picked * (w.to(F64)[..., None] if weights is not None else 1.0)
        ref, mag = terms.sum(1), terms.abs().sum(1)
        got = bsq.expert_combine(y, s.position, weights).to(F64)
        e = (topk + 1) * U * mag  # a product and a sum a term
        assert ((got - ref).abs() <= e + hs * (ref.abs() + e)).all()
    assert torch.equal(bsq.expert_gather_backward(y, s.position), bsq.expert_combine(y, s.position))

    dy, dw = bsq.expert_combine_backward(x, y, s.position, s.slot, w)
    ref = torch.zeros(*y.shape, device="cuda", dtype=F64)
    ref[live] = w.to(F64).reshape(-1)[s.slot[live].long()][:, None] * x.to(F64)[(s.slot[live] // topk).long()]
    assert ((dy.to(F64) - ref).abs() <= hs * ref.abs() * (1 + 2 * U) + U * ref.abs()).all()
    assert (dy[~live] == 0).all()
    terms = picked * x.to(F64)[:, None, :]
    # a lane adds one value in 32 of the row in turn, then 5 shuffles join the lanes
    n = y.shape[1] // 32 + 8 + 8
    assert ((dw.to(F64) - terms.sum(-1)).abs() <= n * U * terms.abs().sum(-1)).all()
    assert (dw[s.position < 0] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [1, 3, 8, 64, 100, 256, 1001, 2048, 5000])
@pytest.mark.parametrize("tokens,topk,experts,align", [(1, 8, 64, 1), (1, 1, 4, 128), (7, 3, 5, 4), (130, 2, 9, 128),
                                                       (515, 8, 32, 1), (64, 17, 40, 1)])
def test_rows(tokens, topk, experts, align, cols, dtype):
    check_rows(*make_rows(tokens, topk, experts, cols, dtype, align, seed=cols))


@pytest.mark.parametrize("kind", ["one", "none"])
def test_rows_of_one_expert_and_of_none(kind):
    check_rows(*make_rows(77, 4, 6, 264, torch.bfloat16, 16, kind=kind))


def test_no_tokens():
    bsq = _bsq()
    s, x, y, w = make_rows(0, 4, 6, 64, torch.bfloat16)
    assert bsq.expert_gather(x, s.position, s.slot).shape == (0, 64)
    assert bsq.expert_combine(y, s.position, w).shape == (0, 64)
    dy, dw = bsq.expert_combine_backward(x, y, s.position, s.slot, w)
    assert dy.shape == (0, 64) and dw.shape == (0, 4)


def test_row_strides_and_odd_addresses():
    s, x, y, w = make_rows(130, 2, 9, 768, torch.bfloat16, 128)

    def inside(t, shift):
        wide = torch.full((t.shape[0], 800), float("nan"), dtype=t.dtype, device="cuda")
        v = wide[:, 8 + shift:776 + shift]
        v.copy_(t)
        return v

    for shift in (0, 1):
        check_rows(s, inside(x, shift), inside(y, shift), w)
    check_rows(s, x[:1].expand(130, 768), y, w)  # the gradient of a broadcast


def test_dropped_choices_and_rows_of_no_slot_are_not_read():
    """NaN in the rows no slot names and in the weights of dropped choices reaches no output."""
    bsq = _bsq()
    s, x, y, w = make_rows(130, 4, 9, 520, torch.bfloat16, 128)
    want = bsq.expert_combine(y, s.position, w), *bsq.expert_combine_backward(x, y, s.position, s.slot, w)
    y[s.slot < 0] = float("nan")
    w[s.position < 0] = float("nan")
    got = bsq.expert_combine(y, s.position, w), *bsq.expert_combine_backward(x, y, s.position, s.slot, w)
    for g, t in zip(got, want):
        assert torch.equal(g, t)


def test_positions_and_slots_outside_the_rows_count_as_dropped():
    bsq = _bsq()
    s, x, y, w = make_rows(50, 4, 9, 256, torch.bfloat16)
    position, slot = s.position.clone(), s.slot.clone()
    position[3, 1], position[4, 0] = y.shape[0], 2 ** 31 - 1
    slot[5], slot[6] = 200, 2 ** 31 - 1
    dropped = torch.where((position < 0) | (position >= y.shape[0]), -1, position).to(torch.int32)
    none = torch.where(slot >= 200, -1, slot).to(torch.int32)
    assert torch.equal(bsq.expert_combine(y, position, w), bsq.expert_combine(y, dropped, w))
    assert torch.equal(bsq.expert_gather(x, position, slot), bsq.expert_gather(x, dropped, none))
    assert bsq.device_status() == 0


def test_there_and_back_is_the_sum_of_the_weights():
    bsq = _bsq()
    ids = torch.stack([torch.randperm(16)[:4] for _ in range(300)]).cuda()
    s = bsq.expert_sort(ids, 16, align=128)
    x = torch.randn(300, 512, device="cuda").to(torch.bfloat16)
    w = torch.full((300, 4), 0.25, device="cuda")
    assert torch.equal(bsq.expert_combine(bsq.expert_gather(x, s.position, s.slot), s.position, w), x)


def test_same_bits_on_another_stream_and_in_a_graph():
    bsq = _bsq()
    s, x, y, w = make_rows(3001, 4, 33, 768, torch.bfloat16, 16)
    ids = make_ids(3001, 4, 33, 0, "outside").cuda()

    def step(stream=None):
        r = bsq.expert_sort(ids, 33, align=16, stream=stream)
        return (*r, bsq.expert_gather(x, r.position, r.slot, stream=stream),
                bsq.expert_combine(y, r.position, w, stream=stream),
                *bsq.expert_combine_backward(x, y, r.position, r.slot, w, stream=stream))

    want = step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = step(st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for t in kept:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, kept):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_gradients_against_differences():
    bsq = _bsq()
    s, x, y, w = make_rows(9, 3, 5, 40, torch.float32, 2)
    dout = torch.randn_like(x)
    dy, dw = bsq.expert_combine_backward(dout, y, s.position, s.slot, w)
    ok = (s.position >= 0)[..., None]
    pos = s.position.clamp(min=0).long()

    def loss(yy, ww):
        return float((torch.where(ok, yy[pos], 0.0) * ww[..., None] * dout.to(F64)[:, None, :]).sum())

    vy, vw = torch.randn_like(y).to(F64), torch.randn_like(w).to(F64)
    y64, w64 = y.to(F64), w.to(F64)
    assert abs(loss(y64 + vy, w64) - loss(y64 - vy, w64) - 2 * float((dy.to(F64) * vy).sum())) < 1e-4
    assert abs(loss(y64, w64 + vw) - loss(y64, w64 - vw) - 2 * float((dw.to(F64) * vw).sum())) < 1e-4


def test_more_than_2_31_elements():
    bsq = _bsq()
    cols = 16384
    tokens = (1 << 31) // cols // 2 + 9
    ids = torch.randint(0, 8, (tokens, 2), device="cuda")
    s = bsq.expert_sort(ids, 8)
    x = torch.randn(64, cols, device="cuda").to(torch.bfloat16).repeat(-(-tokens // 64), 1)[:tokens]
    rows = bsq.expert_gather(x, s.position, s.slot)
    assert rows.numel() > 1 << 31
    for r in (0, 65537, rows.shape[0] - 1):
        assert torch.equal(rows[r], x[int(s.slot[r]) // 2])
    back = bsq.expert_combine(rows, s.position, torch.full((tokens, 2), 0.5, device="cuda"))
    assert torch.equal(back, x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [3, 8, 264, 1001, 1500])
@pytest.mark.parametrize("topk,experts,align", [(1, 4, 1), (2, 16, 128), (3, 9, 16), (4, 300, 1), (8, 8, 64), (11, 40, 1),
                                                (40, 64, 4)])
def test_rows_of_many_tokens(topk, experts, align, cols, dtype):
    """Enough tokens for the kernels that take a token with all its choices."""
    check_rows(*make_rows(2311, topk, experts, cols, dtype, align, seed=cols + topk))


def test_pairs_that_do_not_name_each_other_count_as_none_for_many_tokens():
    bsq = _bsq()
    s, x, y, w = make_rows(2500, 4, 9, 256, torch.bfloat16)
    position, slot = s.position.clone(), s.slot.clone()
    n = position.numel()
    position[3, 1], position[4, 0] = y.shape[0], 2 ** 31 - 1
    slot[5], slot[6] = n, 2 ** 31 - 1
    slot[7] = slot[8]                       # two rows that name one slot
    position[20, 2] = position[21, 2]       # two slots that name one row
    rows = bsq.expert_gather(x, position, slot)
    flat = position.reshape(-1)
    agree = (slot >= 0) & (slot < n)
    agree &= flat[slot.clamp(0, n - 1).long()] == torch.arange(slot.numel(), device="cuda")
    want = torch.where(agree[:, None], x[(slot.clamp(0, n - 1) // 4).long()], torch.zeros_like(rows))
    assert torch.equal(rows, want)
    dy, _ = bsq.expert_combine_backward(x, y, position, slot, w)
    assert (dy[~agree] == 0).all()
    few = bsq.expert_gather(x[:1000], position[:1000].contiguous(), slot)
    agree &= slot < 4000
    assert torch.equal(few, torch.where(agree[:, None], want, torch.zeros_like(want)))
    assert bsq.device_status() == 0
