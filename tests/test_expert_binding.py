"""The expert operators' binding on the host: what it does before a call reaches the library."""
from types import SimpleNamespace

import pytest
import torch

from row_wise_softmax_warp_gb300 import binding


def test_a_stream_of_another_device_is_refused():
    """Made current it would switch the device too, and the call would have gone to a stream that nobody named."""
    tensor = SimpleNamespace(device=torch.device("cuda", 0))
    for other in (torch.device("cuda", 1), torch.device("cpu")):
        with pytest.raises(ValueError, match="stream is on"):
            binding._Placed(tensor, SimpleNamespace(device=other))
    binding._Placed(tensor, None)


def test_room_for_shifted_matrices():
    """Bytes for what starts off a boundary; what the library's functions count already is not counted twice."""
    at = lambda address: SimpleNamespace(data_ptr=lambda: address)  # noqa: E731
    assert binding._shifted_room((at(4096), 10, 32), (at(8192), 5, 64)) == 0
    assert binding._shifted_room((at(4098), 10, 32), (at(8192), 5, 64)) == 10 * 32 + 512
    assert binding._shifted_room((at(4098), 10, 32), (at(8194), 5, 64)) == 10 * 32 + 5 * 64 + 1024
    assert binding._shifted_room((at(4098), 10, 34)) == 0
