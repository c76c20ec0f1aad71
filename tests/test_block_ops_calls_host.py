"""How the functions around the linear layers hand a call on, without a GPU: streams, devices and the
C++ host side are stood in for."""
import pytest
import torch


@pytest.fixture(scope="module")
def bsq():
    import __graft_entry__

    __graft_entry__.build()
    import block_scaled_precision_bsq_gb300 as b

    return b


def test_a_stream_handle_of_zero_is_the_default_stream(bsq, monkeypatch):
    """torch.cuda.default_stream().cuda_stream is 0, and 0 is the library's legacy default stream too."""
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    assert bsq._torch_stream(0) == "default"
    assert bsq._torch_stream(1 << 40) == ("external", 1 << 40)
