"""Gradients of the layer norm of values far from zero (needs a B200).

x - m of values close to the mean is exact in fp32, or off by u = 2^-24 of itself, and so is its product with r: the
normalised value xh is within 4 u |xh| however far the mean lies, and the sums follow as in
tests/test_gpu_layer_norm.py: n terms in any order within n u of the sum of their sizes, each result rounded once to
its type. Rows and groups are few and narrow (or the other one is), so that n u hides nothing of the offset's size."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

# lane teams, block teams, a warp's worth, four vectors a thread, rows that no vector divides, rows too wide
SHAPES = [(6, 4, 64), (5, 3, 24), (2, 1, 2688), (2, 1, 16384), (4, 1, 33), (2, 1, 40000)]


@pytest.mark.parametrize("rows,groups,width", SHAPES)
@pytest.mark.parametrize("act,offset", [("f32", 1000.0), ("f32", -30000.0), ("bf16", 100.0)])
def test_gradients_far_from_zero(rows, groups, width, act, offset):
    gen = torch.Generator().manual_seed(width)
    C, a = groups * width, torch.bfloat16 if act == "bf16" else torch.float32
    x = (offset + torch.randn(rows, C, generator=gen)).to(a).cuda()
    dy = torch.randn(rows, C, generator=gen).to(a).cuda()
    w = (1 + 0.3 * torch.randn(C, generator=gen)).cuda()
    _, mean, rstd = sm.layer_norm(x, w, None, groups=groups)
    dx, dw, db = sm.layer_norm_backward(dy, x, w, mean, rstd, groups=groups)

    shape = (rows, groups, width)
    xd, gd, wd = x.double().view(shape), dy.double().view(shape), w.double().view(1, groups, width)
    m, r = mean.double()[..., None], rstd.double()[..., None]
    xh, dh = (xd - m) * r, gd * wd
    m1, m2 = dh.mean(-1, keepdim=True), (dh * xh).mean(-1, keepdim=True)
    ref = r * (dh - m1 - xh * m2)
    a1, a2 = dh.abs().mean(-1, keepdim=True), (dh * xh).abs().mean(-1, keepdim=True)
    exh = 4 * U * xh.abs()
    e = r * ((width + 8) * U * (a1 + xh.abs() * a2) + 8 * U * (dh.abs() + a1 + xh.abs() * a2) + exh * a2
             + xh.abs() * (dh.abs() * exh).mean(-1, keepdim=True))
    e = e + torch.finfo(a).eps / 2 * (ref.abs() + e)
    assert bool(((dx.double().view(shape) - ref).abs() <= e).all()), float(((dx.double().view(shape) - ref).abs() / e).max())
    ew = ((rows + 8) * U * (gd * xh).abs().sum(0) + (gd.abs() * exh).sum(0)).flatten()
    got = (dw.double() - (gd * xh).sum(0).flatten()).abs()
    assert bool((got <= ew + 1e-30).all()), float((got / (ew + 1e-30)).max())
    assert bool(((db.double() - gd.sum(0).flatten()).abs() <= ((rows + 8) * U * gd.abs().sum(0)).flatten()).all())
