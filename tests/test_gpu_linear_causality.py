"""NaN and infinities of one token reach the tokens that its formula names, and no others (needs a B200): forwards
those behind it, in the gradients those before it."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import dims, make

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", (2, 300, 2, 2, 64, 64)), ("bf16", (1, 300, 2, 1, 128, 128)), ("bf16", (2, 260, 2, 2, 64, 128)),
          ("bf16", (1, 389, 2, 2, 128, 64)), ("f32", (2, 60, 2, 2, 32, 16)), ("bf16", (2, 7, 2, 2, 64, 64))]


def finite(t):
    return t.isfinite()


@pytest.mark.parametrize("act,shape", SHAPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", [0.0, 0.4, 0.5, 0.999])
def test_forward(act, shape, bad, where):
    """A few of v's columns at one token: those columns of o from that token on, and those rows of the state."""
    b, L, H, G, dk, dv = shape
    d = dims(*shape, act)
    x = make(*shape, act, seed=L)
    t, cols = int(where * L), [0, 3, dv - 1]
    v = x["v"].clone()
    v.view(b, L, G, dv)[0, t, :, cols] = bad
    (o, fs), (co, cs) = (sm.linear_prefill(d, x["q"], x["k"], w, x["log_decay"], x["init"]) for w in (v, x["v"]))
    o, co = o.view(b, L, H, dv), co.view(b, L, H, dv)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, t:, :, cols] = True
    assert torch.equal(o[~hit], co[~hit]) and not bool(finite(o[hit]).any()) and bool(finite(co).all())
    hit = torch.zeros_like(fs, dtype=torch.bool)
    hit[0, :, cols] = True
    assert torch.equal(fs[~hit], cs[~hit]) and not bool(finite(fs[hit]).any())


# a NaN at token t of each operand: the gradients that it reaches at t itself, before it and behind it
REACH = {"q": {"k": "to", "v": "to"}, "k": {"q": "from", "v": "at"}, "v": {"q": "from", "k": "at"},
         "do": {"q": "at", "k": "to", "v": "to"}}


@pytest.mark.parametrize("act,shape", SHAPES)
@pytest.mark.parametrize("operand", list(REACH))
@pytest.mark.parametrize("where", [0.0, 0.4, 0.5, 0.999])
def test_backward(act, shape, operand, where):
    b, L, H, G, dk, dv = shape
    d = dims(*shape, act)
    x = make(*shape, act, seed=L + 1)
    t = int(where * L)
    y = dict(x, **{operand: x[operand].clone()})
    y[operand][0, t, 3::16] = float("nan")
    g, c = (sm.linear_backward(d, z["q"], z["k"], z["v"], z["log_decay"], z["do"], z["init"], z["dfinal"]) for z in (y, x))
    for n in ("q", "k", "v"):
        hit = torch.zeros(b, L, dtype=torch.bool, device="cuda")
        at = {"to": slice(None, t + 1), "from": slice(t, None), "at": slice(t, t + 1), None: slice(0, 0)}[REACH[operand].get(n)]
        hit[0, at] = True
        assert torch.equal(g[n][~hit], c[n][~hit]) and bool(finite(c[n]).all()), n
        if bool(hit.any()):
            assert not bool(finite(g[n][hit]).all(-1).any()), n
