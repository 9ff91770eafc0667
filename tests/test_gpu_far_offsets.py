"""Linear attention and layer norm where an element's offset passes 2^31 (needs a B200 and some 12 GB):
slots far into a cache of states, rows far apart. The same call on compact copies gives the same bits."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import make

pytestmark = pytest.mark.gpu

H, D, FAR = 2, 128, 70000          # 70000 slots of 2 x 128 x 128, or rows of 70000 elements


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_slots_far_into_the_cache(act):
    cache = torch.empty(FAR, H, D, D, device="cuda")
    lens, slots = [3, 200, 700], [FAR - 1, FAR - 2, 1]
    near = torch.arange(3, dtype=torch.int32, device="cuda")
    far = torch.tensor(slots, dtype=torch.int32, device="cuda")
    x = make(1, sum(lens), H, H, D, D, act, seed=1)
    small = torch.randn(3, H, D, D, generator=torch.Generator().manual_seed(2)).cuda()
    cache[far.long()] = small
    cu = torch.tensor([0, 3, 203, 903], dtype=torch.int32, device="cuda")
    d, one = (sm.LinearDims(3, n, H, H, D, D, act=act) for n in (sum(lens), 1))
    out = []
    for state, slot in ((small, near), (cache, far)):
        q, k, v = (x[n][0] for n in ("q", "k", "v"))
        o = sm.linear_prefill_varlen(d, cu, slot, None, q, k, v, x["log_decay"], state)
        out.append([o, sm.linear_decode_step(one, q[:3], k[:3], v[:3], x["log_decay"], state, slot), state[slot.long()]])
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_rows_far_apart(act):
    L = 31000                      # 31000 x 70000 > 2^31
    x = make(1, L, H, H, D, D, act, seed=3)
    wide = torch.empty(1, L, FAR, dtype=x["q"].dtype, device="cuda")
    W = H * D
    part = {n: wide[:, :, 64 * i * 8:64 * i * 8 + W] for i, n in enumerate(("q", "k", "v", "do"))}
    for n, t in part.items():
        t.copy_(x[n])
    d = sm.LinearDims(1, L, H, H, D, D, scale=D ** -0.5, act=act)
    o, fs = sm.linear_prefill(d, x["q"], x["k"], x["v"], x["log_decay"], x["init"])
    far = wide[:, :, FAR - W:]
    _, fs2 = sm.linear_prefill(d, part["q"], part["k"], part["v"], x["log_decay"], x["init"], out=(far, torch.empty_like(fs)))
    assert torch.equal(far, o) and torch.equal(fs2, fs)
    near = sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"])
    wide_g = sm.linear_backward(d, part["q"], part["k"], part["v"], x["log_decay"], part["do"], x["init"], x["dfinal"])
    for n in near:
        assert torch.equal(near[n], wide_g[n])
    w = torch.ones(W, device="cuda")
    for groups in (1, H):
        y, m, r = sm.layer_norm(x["q"], w, None, groups=groups)
        y2, m2, r2 = sm.layer_norm(part["q"], w, None, groups=groups, out=far)
        assert torch.equal(y, far) and torch.equal(m, m2) and torch.equal(r, r2)
        for a, b in zip(sm.layer_norm_backward(x["do"], x["q"], w, m, r, groups=groups),
                        sm.layer_norm_backward(part["do"], part["q"], w, m2, r2, groups=groups)):
            assert torch.equal(a, b)
