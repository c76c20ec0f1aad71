"""block_norm and block_norm_backward where offsets and clusters reach their limits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsq():
    import block_scaled_precision_bsq_gb300 as bsq

    return bsq


@pytest.mark.parametrize("off", [0, 1])
def test_blocks_of_rows_at_the_limit_of_32_bit_offsets(off):
    """300000 rows of 65536 columns: 9 clusters would have taken blocks of 33334 rows, more than 2^31 elements.
    One row repeated (stride 0) stands for all inputs; off: by vectors, and element by element."""
    bsq = _bsq()
    rows, cols = 300000, 65536
    g = torch.Generator(device="cuda").manual_seed(off)
    x, dy = (torch.randn(cols + 8, device="cuda", generator=g).to(torch.bfloat16)[off:cols + off].expand(4, cols)
             for _ in range(2))
    f = bsq.block_norm(None, x, kind="rms")
    few = bsq.block_norm_backward(None, dy, x, None, f.stats, kind="rms").dx
    assert torch.equal(few, few[:1].expand(4, cols))
    stats = f.stats[:1].expand(rows, 4).contiguous()
    dx = bsq.block_norm_backward(None, dy[:1].expand(rows, cols), x[:1].expand(rows, cols), None, stats, kind="rms").dx
    for at in range(0, rows, 10000):
        assert torch.equal(dx[at:at + 10000], few[:1].expand(10000, cols)), at
    assert bsq.device_status() == 0


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("cols", [4089, 4090, 4095, 8191, 65521, 65529, 65530, 65532, 65535])
def test_widths_whose_first_vector_reaches_over_the_row(cols, kind):
    """Just below the widths of one CTA, of a cluster of 2 and of the largest cluster."""
    from test_gpu_block_norm import Case, run

    run(Case(5, cols, kind, torch.bfloat16, seed=cols))
    run(Case(40, cols, kind, torch.bfloat16, groups=2, bias=False, seed=cols))


@pytest.mark.parametrize("cols", [4092, 4093, 4095, 32765, 32767])
def test_fp32_widths_whose_first_vector_reaches_over_the_row(cols):
    from test_gpu_block_norm import Case, run

    run(Case(5, cols, "layer", torch.float32, torch.float32, seed=cols))
    run(Case(40, cols, "rms", torch.float32, torch.float32, groups=2, bias=False, seed=cols))


def test_row_numbers_at_the_limit_of_32_bits():
    """2^31 - 2 rows of one column, a gate for each 62: the last gates' rows lie within a CTA's step of 2^31. Without
    a post norm dh is dx_out * gate."""
    bsq = _bsq()
    rows, each = (1 << 31) - 2, 62
    groups = rows // each
    assert groups * each == rows
    g = torch.Generator(device="cuda").manual_seed(3)
    gate = torch.randn(groups, 1, device="cuda", generator=g).to(torch.bfloat16)
    one = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    dh = torch.full((rows, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    a = bsq.BlockNormGradArgs(kind=bsq.NORM_RMS, flags=0, rows=rows, cols=1, gate_groups=groups, residual_scale=1.0,
                              dx_out=p(one), dx_out_stride=1, gate=p(gate), dh=p(dh))
    assert bsq.bsq_block_norm_backward(a) == bsq.OK
    got, step = dh.view(groups, each), 1 << 22
    for at in range(0, groups, step):
        assert torch.equal(got[at:at + step], gate[at:at + step].expand(-1, each)), at
    assert bsq.device_status() == 0
