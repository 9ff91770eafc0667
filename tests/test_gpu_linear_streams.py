"""Which stream and device the calls of linear attention and layer norm run on (needs a B200)."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import dims, make

pytestmark = pytest.mark.gpu


def spy(monkeypatch, name):
    """The stream handles that the library's entry `name` is called with."""
    seen, entry = [], getattr(sm.load_library(), name)

    def call(*args):
        seen.append(args[-1])
        return entry(*args)

    monkeypatch.setattr(sm.load_library(), name, call, raising=False)
    return seen


@pytest.mark.parametrize("kind", ["none", "handle", "zero", "stream"])
@pytest.mark.parametrize("current", ["default", "other"])
def test_the_stream_given_is_the_one_used(monkeypatch, kind, current):
    """A handle as an integer is that stream; 0 is the default stream whichever is current."""
    given, here = torch.cuda.Stream(), torch.cuda.Stream()
    stream, want = {"none": (None, None), "handle": (given.cuda_stream, given.cuda_stream), "zero": (0, 0),
                    "stream": (given, given.cuda_stream)}[kind]
    d = dims(1, 20, 2, 2, 64, 64, "bf16")
    x = make(1, 20, 2, 2, 64, 64, "bf16", seed=1)
    torch.cuda.synchronize()
    with torch.cuda.stream(here if current == "other" else torch.cuda.default_stream()):
        if want is None:
            want = torch.cuda.current_stream().cuda_stream
        a = spy(monkeypatch, "ssd_mixer_linear_prefill")
        sm.linear_prefill(d, x["q"], x["k"], x["v"], x["log_decay"], stream=stream)
        b = spy(monkeypatch, "ssd_mixer_layer_norm")
        sm.layer_norm(x["q"], stream=stream)
        assert a == [want] and b == [want]
    torch.cuda.synchronize()


def test_a_refused_stream_leaves_the_current_device_and_stream():
    x = torch.zeros(2, 64, device="cuda")
    before = torch.cuda.current_device(), torch.cuda.current_stream()
    for bad in ("a name", object()):
        with pytest.raises((TypeError, ValueError)):
            sm.layer_norm(x, stream=bad)
    assert (torch.cuda.current_device(), torch.cuda.current_stream()) == before
