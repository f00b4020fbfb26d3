"""A stream given to a slot call belongs to the state's device (no GPU needed)."""
import pytest
import torch

from quantized_recurrent_state_amd import slots


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Stream:                            # what the check reads of a torch stream
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device("cuda", index), 123

    class Current:
        def __init__(self, stream):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *exc):
            pass

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", Current)
    calls = []
    assert slots._on_device(0, Stream(0), lambda s: calls.append(s) or 7) == 7
    with pytest.raises(ValueError):
        slots._on_device(0, Stream(1), calls.append)
    assert calls == [123]
