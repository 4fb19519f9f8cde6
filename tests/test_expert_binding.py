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
