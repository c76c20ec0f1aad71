"""The injected stall of block_norm_backward's cluster kernel on RMS norms, and one that is never reached."""
import pytest
import torch

from test_gpu_block_norm import Case, check

pytestmark = pytest.mark.gpu

PAST = 100000  # rows of a gate row's in one cluster: never so many here


def _backward(bsq, c, f):
    return bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dtype,cols,off", [(torch.bfloat16, 8192, 0), (torch.bfloat16, 9001, 0),
                                            (torch.bfloat16, 8192, 1), (torch.float32, 5000, 0)])
def test_a_stall_behind_the_last_row_changes_nothing(dtype, cols, off, bias, kind):
    import block_scaled_precision_bsq_gb300 as bsq

    c = Case(300, cols, kind, dtype, bias=bias, groups=2, seed=cols)
    if off:  # rows that are read element by element
        wide = torch.zeros(300, cols + 8, dtype=dtype, device="cuda")
        wide[:, 1:cols + 1] = c.dy
        c.dy = wide[:, 1:cols + 1]
    f = bsq.block_norm(c.h, c.x, eps=c.eps, **c.kw())
    assert bsq.bsq_test_inject_stall(bsq.KERNEL_NORM, PAST, 1_000_000_000) == bsq.OK
    r = _backward(bsq, c, f)
    assert bsq.device_status() == bsq.OK
    want = c.backward(f.x_out, f.stats)
    for name, given in (("dx", True), ("dh", True), ("dpost_weight", c.w1), ("dpost_bias", c.b1), ("dgate", c.gate),
                        ("dpre_weight", c.w2), ("dpre_bias", c.b2)):
        if given is not None:
            check(getattr(r, name), want[name], name)


@pytest.mark.parametrize("after", [0, 2])
@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 8192), (torch.bfloat16, 9001), (torch.float32, 5000)])
def test_a_stall_of_an_rms_norm_reports_a_timeout(dtype, cols, after):
    import block_scaled_precision_bsq_gb300 as bsq

    c = Case(700, cols, "rms", dtype, bias=False)
    f = bsq.block_norm(c.h, c.x, **c.kw())
    want = _backward(bsq, c, f)
    assert bsq.device_status() == bsq.OK
    assert bsq.bsq_test_inject_stall(bsq.KERNEL_NORM, after, 2_000_000) == bsq.OK
    _backward(bsq, c, f)
    assert bsq.device_status() == bsq.ERR_TIMEOUT
    for a, b in zip(_backward(bsq, c, f), want):
        assert a is None and b is None or torch.equal(a, b)
    assert bsq.device_status() == bsq.OK
