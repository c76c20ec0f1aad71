"""Sizes of the expert rows that no test allocates, refused before any CUDA call."""
import pytest

P = 1 << 20  # a 16-byte aligned dummy address: never dereferenced on these paths


@pytest.fixture(scope="module")
def bsq():
    import __graft_entry__

    __graft_entry__.build()
    import block_scaled_precision_bsq_gb300 as b

    return b


@pytest.mark.parametrize("cols", [(1 << 30) + 1, (1 << 31) - 256, (1 << 31) - 1])
def test_rows_whose_columns_pass_a_lanes_counter_are_refused(bsq, cols):
    """A lane counts a row's elements in 32 bits, in steps of up to 256: near 2^31 columns the count wrapped."""
    for flags in (0, bsq.FLAG_SRC_F32):
        assert bsq.bsq_expert_gather(flags, P, cols, P, P, 4, 2, cols, 8, P) == bsq.ERR_SHAPE
        assert bsq.bsq_expert_combine(flags, P, cols, P, P, 4, 2, cols, 8, P) == bsq.ERR_SHAPE
        assert bsq.bsq_expert_combine_backward(flags, P, cols, P, cols, P, P, P, 4, 2, cols, 8, P, P) == bsq.ERR_SHAPE
