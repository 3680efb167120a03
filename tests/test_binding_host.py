"""What the binding decides on the host (no GPU)."""
from types import SimpleNamespace

import pytest

from bidirectional_mamba_selective_amd import _lib


def test_a_stream_of_another_device_is_refused():
    """The kernels would run on the stream's device with addresses of the tensors' device."""
    torch = pytest.importorskip("torch")
    dev = [torch.device("cuda", i) for i in range(2)]
    stream = SimpleNamespace(device=dev[1], cuda_stream=0x1230)
    assert _lib._stream(stream, dev[1]) == 0x1230
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        _lib._stream(stream, dev[0])
