"""The binding's choice of device and stream, with torch.cuda's contexts replaced (CPU only)."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm


class _Context:
    entered = 0

    def __init__(self, *args):
        pass

    def __enter__(self):
        _Context.entered += 1

    def __exit__(self, *exc):
        _Context.entered -= 1


@pytest.mark.parametrize("bad", ["a name", object(), None])
def test_a_refused_stream_enters_no_device(monkeypatch, bad):
    """Tensors on another device than the current one, and a stream that is none or is on the current one."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", _Context)
    monkeypatch.setattr(torch.cuda, "stream", _Context)
    if bad is None:
        class Stream:
            device, cuda_stream = torch.device("cuda", 0), 1
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        bad = Stream()
    _Context.entered = 0
    with pytest.raises((TypeError, ValueError)):
        with sm._On(torch.device("cuda", 1), bad):
            pass
    assert _Context.entered == 0
