"""A NaN among the decays of linear attention comes out as NaN, in its own head alone (needs a B200)."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import dims, make

pytestmark = pytest.mark.gpu

# tensor cores (one block, several, cut into segments), CUDA cores, short rows of both
SHAPES = [("bf16", (2, 100, 3, 3, 64, 64)), ("bf16", (1, 400, 3, 3, 128, 64)), ("bf16", (1, 4000, 2, 2, 64, 128)),
          ("f32", (2, 90, 3, 3, 32, 16)), ("f32", (1, 1500, 2, 2, 64, 64)), ("bf16", (2, 5, 2, 2, 64, 64)), ("f32", (2, 5, 2, 2, 16, 32))]


@pytest.mark.parametrize("act,shape", SHAPES)
def test_nan_decay(act, shape):
    b, L, H, G, dk, dv = shape
    d, one = dims(*shape, act), dims(b, 1, H, G, dk, dv, act)
    x = make(*shape, act, seed=L)
    bad = x["log_decay"].clone()
    bad[1] = float("nan")

    def calls(decay):
        o, fs = sm.linear_prefill(d, x["q"], x["k"], x["v"], decay, x["init"])
        packed = dims(b, b * L, H, G, dk, dv, act)
        state = x["init"].clone()
        cu = torch.arange(0, b * L + 1, L, dtype=torch.int32, device="cuda")
        po = sm.linear_prefill_varlen(packed, cu, None, None, *(x[n].view(b * L, -1) for n in ("q", "k", "v")), decay, state)
        step = x["init"].clone()
        so = sm.linear_decode_step(one, x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], decay, step)
        g = sm.linear_backward(d, x["q"], x["k"], x["v"], decay, x["do"], x["init"], x["dfinal"])
        # the last token's dk and dv are those of the state's gradient before any decay
        return {"o": o.view(b, L, H, dv), "state": fs.transpose(0, 1), "packed o": po.view(b, L, H, dv),
                "packed state": state.transpose(0, 1), "decode o": so.view(b, 1, H, dv), "decode state": step.transpose(0, 1),
                "dq": g["q"].view(b, L, H, dk), "dk": g["k"].view(b, L, H, dk)[:, :-1], "dv": g["v"].view(b, L, H, dv)[:, :-1],
                "dinit": g["init_state"].transpose(0, 1)}

    clean, got = calls(x["log_decay"]), calls(bad)
    for n, t in got.items():
        heads = t if "state" in n or n == "dinit" else t.permute(2, 0, 1, 3)
        ref = clean[n] if heads is t else clean[n].permute(2, 0, 1, 3)
        assert bool(heads[1].isnan().all()), n
        assert torch.equal(heads[::2], ref[::2]) and not bool(ref.isnan().any()), n
