"""Block norms whose matrices or parameters do not allow 16-byte vectors: element by element, within a CTA and
across a cluster, under one gate row and several."""
import pytest
import torch

from test_gpu_block_norm import Case, run

pytestmark = pytest.mark.gpu

PARAMS = ("w1", "b1", "gate", "w2", "b2")
MATRICES = ("h", "x", "dxo", "dy")


def off_by_one(t):
    """The same values one element behind a 16-byte boundary."""
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = room[1:].view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 16 != 0 and v.is_contiguous()
    return v


def odd_rows(t, shift):
    """The same values as rows of a wider matrix of NaN, `shift` elements behind a 16-byte boundary."""
    room = torch.full((t.shape[0], t.shape[1] + 24), float("nan"), dtype=t.dtype, device=t.device)
    v = room[:, 8 + shift:8 + shift + t.shape[1]]
    v.copy_(t)
    return v


@pytest.mark.parametrize("name", PARAMS)
@pytest.mark.parametrize("params", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups", [1, 3])
def test_one_parameter_at_an_odd_address(groups, params, name):
    c = Case(39, 768, "layer", torch.bfloat16, params, groups=groups, seed=7)
    setattr(c, name, off_by_one(getattr(c, name)))
    run(c)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("dtype,params,cols", [
    (torch.bfloat16, torch.bfloat16, 64), (torch.bfloat16, torch.float32, 1024), (torch.bfloat16, torch.bfloat16, 4096),
    (torch.bfloat16, torch.float32, 8192), (torch.bfloat16, torch.bfloat16, 20480), (torch.bfloat16, torch.float32, 65536),
    (torch.float32, torch.bfloat16, 768), (torch.float32, torch.float32, 5120), (torch.float32, torch.float32, 16384),
    (torch.float32, torch.bfloat16, 32768)])
def test_all_parameters_at_odd_addresses(dtype, params, cols, groups, kind):
    """From 4096 columns on (backward), from 16384 bf16 or 8192 fp32 on (forward) a row is held by a cluster."""
    for rows in (4, 324):
        c = Case(rows, cols, kind, dtype, params, groups=groups, bias=kind == "layer", seed=cols)
        for name in PARAMS:
            if getattr(c, name) is not None:
                setattr(c, name, off_by_one(getattr(c, name)))
        run(c)


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 256), (torch.bfloat16, 5000), (torch.bfloat16, 9001),
                                        (torch.bfloat16, 20000), (torch.bfloat16, 65535), (torch.float32, 264),
                                        (torch.float32, 4101), (torch.float32, 12289), (torch.float32, 32768)])
def test_matrices_of_unlike_alignment(dtype, cols, groups):
    """Each matrix at an offset of its own inside 16 bytes."""
    for rows, kind in ((4, "layer"), (324, "rms")):
        c = Case(rows, cols, kind, dtype, groups=groups, bias=kind == "layer", seed=cols)
        for shift, name in enumerate(MATRICES):
            setattr(c, name, odd_rows(getattr(c, name), shift))
        run(c)


@pytest.mark.parametrize("rows,cols", [(12, 1001), (320, 1023), (12, 9001), (160, 5001)])
@pytest.mark.parametrize("group_rows", [1, 2])
def test_many_gates_of_fewer_rows_than_alignment_classes(rows, cols, group_rows):
    """From 32 gates on these are read element by element, few gates by vectors."""
    for dtype in (torch.bfloat16, torch.float32):
        run(Case(rows, cols, "layer", dtype, torch.float32, groups=rows // group_rows, seed=rows))


def test_unaligned_rows_of_nan_do_not_reach_their_neighbours():
    import block_scaled_precision_bsq_gb300 as bsq

    for cols in (768, 9001):
        c = Case(40, cols, "layer")
        for shift, name in enumerate(MATRICES):
            setattr(c, name, odd_rows(getattr(c, name), shift))
        f = bsq.block_norm(c.h, c.x, **c.kw())
        r = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
        for t in (c.h, c.x, c.dxo, c.dy):
            t[3] = float("nan")
        f2 = bsq.block_norm(c.h, c.x, **c.kw())
        r2 = bsq.block_norm_backward(c.dxo, c.dy, f2.x_out, c.h, f2.stats, **c.kw())
        rest = [i for i in range(40) if i != 3]
        for a, b in ((f.x_out, f2.x_out), (f.y, f2.y), (f.stats, f2.stats), (r.dx, r2.dx), (r.dh, r2.dh)):
            assert torch.equal(a[rest], b[rest])
        assert f2.y[3].isnan().all() and r2.dx[3].isnan().all()
    assert bsq.device_status() == 0
