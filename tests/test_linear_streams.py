"""A stream of another device is refused before anything is queued on it."""
import types

import pytest

torch = pytest.importorskip("torch")
from gated_deltanet_recurrence_delta_amd import linear  # noqa: E402


def test_a_stream_of_another_device_is_refused():
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    stream = types.SimpleNamespace(device=there, cuda_stream=77)
    assert linear._raw_stream(there, stream) == 77
    with pytest.raises(ValueError, match="stream must be one of cuda:0"):
        linear._raw_stream(here, stream)
