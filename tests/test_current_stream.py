"""The binding's current stream, on the CPU: torch's quick functions where this torch has them,
and the public call where it does not."""
import types

import pytest

from bidirectional_mamba_state_amd import bdssm

torch = pytest.importorskip("torch")


@pytest.fixture
def device(monkeypatch):
    """A device 1 whose current stream is 0x1000, or 0x2000 as the public call has it."""
    monkeypatch.setattr(bdssm, "_current", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0x2000))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x1000 * d, raising=False)
    return monkeypatch


def test_quick_functions(device):
    assert bdssm._stream(None) == 0x1000 == bdssm._stream(None)


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_public_call_where_a_quick_function_is_missing(device, missing):
    device.delattr(torch._C, missing)
    assert bdssm._stream(None) == 0x2000 == bdssm._stream(None)


def test_a_given_stream_is_used_as_it_is(device):
    assert bdssm._stream(0) == 0 and bdssm._stream(7) == 7
    assert bdssm._stream(types.SimpleNamespace(cuda_stream=9)) == 9
