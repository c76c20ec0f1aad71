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
