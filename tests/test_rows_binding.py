"""The row operators' binding, host only: streams and the argument checks' library."""
from types import SimpleNamespace

import pytest

import token_choice_routing_amd as tcr


def test_stream_of_another_device_is_refused():
    """The call's tensors are on the current device, so its stream has to be as well."""
    assert tcr._row_stream(SimpleNamespace(cuda_stream=16, device_index=0), 0) == 16
    assert tcr._row_stream(SimpleNamespace(cuda_stream=16), 0) == 16  # a handle of another library
    assert tcr._row_stream(32, 1) == 32
    with pytest.raises(ValueError, match="stream: expected one of the current device"):
        tcr._row_stream(SimpleNamespace(cuda_stream=16, device_index=1), 0)
