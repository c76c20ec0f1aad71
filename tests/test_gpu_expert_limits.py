"""expert_sort at its largest capacity."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_segments_that_end_just_below_2_31_rows():
    """8 experts with segments of 2^28 - 1 rows: the last ends 8 rows before 2^31."""
    import block_scaled_precision_bsq_gb300 as bsq

    align = (1 << 28) - 1
    ids = torch.tensor([[3, 0, 7, 1, 2, 6, 5, 4]], device="cuda")
    s = bsq.expert_sort(ids, 8, align=align)
    assert s.slot.numel() == 8 * align
    assert s.counts.tolist() == [1] * 8 and s.offsets.tolist() == [e * align for e in range(9)]
    assert s.position.tolist() == [[e * align for e in ids[0].tolist()]]
    assert s.slot[s.position[0].long()].tolist() == list(range(8))
    s.slot[s.position[0].long()] = -1
    assert all(int(part.max()) == -1 and int(part.min()) == -1 for part in s.slot.split(1 << 28))
    assert bsq.device_status() == 0
