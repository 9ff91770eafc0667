"""GPU parity of the grouped layer norm and its gradients with their fp64 form (needs a B200).

Bounds, with u = 2^-24: sums of n fp32 terms in any order are off by at most n u times the sum of the
terms' sizes. mean: n u mean|x|. The variance around the mean gives rstd within (2 n + 8) u relative
when the spread is not far below the values (else the mean's error adds (n u mean|x| rstd)). y follows
by the chain of products; each result is rounded once more to its type, finfo.eps / 2 of its value."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import norm64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

# (leading shape, groups, width): one element, odd widths, head norms, one wave, wide rows
SHAPES = [((1,), 1, 1), ((3,), 1, 7), ((2, 5), 4, 64), ((9,), 3, 16), ((7,), 2, 100), ((65,), 1, 333), ((4, 33), 8, 128),
          ((300,), 1, 2688), ((5,), 1, 4096), ((3,), 1, 8192), ((2,), 1, 16384), ((2,), 1, 20001), ((1000,), 6, 32), ((2,), 2, 40000),
          ((515,), 1, 1024), ((40,), 5, 520)]


def make(lead, groups, width, act, seed, offset=1.0):
    gen = torch.Generator().manual_seed(seed)
    C = groups * width
    a = torch.bfloat16 if act == "bf16" else torch.float32
    x = (torch.randn(*lead, C, generator=gen) * 2 + offset).to(a).cuda()
    dy = torch.randn(*lead, C, generator=gen).to(a).cuda()
    w, b = (1 + 0.3 * torch.randn(C, generator=gen)).cuda(), torch.randn(C, generator=gen).cuda()
    return x, dy, w, b


def check_norm(x, w, b, groups, eps, y, mean, rstd):
    xd = x.double()
    W = x.shape[-1] // groups
    ry, rm, rr = norm64(xd, None if w is None else w.double(), None if b is None else b.double(), groups, eps)
    xs = xd.abs().unflatten(-1, (groups, W)).mean(-1)
    em = (W + 4) * U * xs
    assert bool(((mean.double() - rm).abs() <= em + 1e-30).all())
    er = ((2 * W + 16) * U + (em * rr) ** 2 + 2 * em * U * rr) * rr
    assert bool(((rstd.double() - rr).abs() <= er).all())
    half = torch.finfo(x.dtype).eps / 2
    c = (xd.unflatten(-1, (groups, W)) - rm[..., None]).abs()
    ey = (c * er[..., None] + (em * rr)[..., None] + 6 * U * (c * rr[..., None])).flatten(-2)
    if w is not None:
        ey = ey * w.double().abs()
    ey = ey + 2 * U * (0 if b is None else b.double().abs()) + half * (ry.abs() + ey)
    assert bool(((y.double() - ry).abs() <= ey).all()), float(((y.double() - ry).abs() / ey).max())


@pytest.mark.parametrize("lead,groups,width", SHAPES)
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_forward(lead, groups, width, act):
    x, _, w, b = make(lead, groups, width, act, seed=width)
    check_norm(x, w, b, groups, 1e-5, *sm.layer_norm(x, w, b, groups=groups))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(act, weight, bias):
    x, _, w, b = make((31,), 2, 96, act, seed=1)
    w, b = w if weight else None, b if bias else None
    check_norm(x, w, b, 2, 1e-3, *sm.layer_norm(x, w, b, groups=2, eps=1e-3))


@pytest.mark.parametrize("groups,width", [(1, 512), (1, 1001), (4, 64)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_strided_rows_odd_offsets_and_in_place(groups, width, act):
    """Rows with gaps, starting at an address that is not 16-byte aligned; y over x."""
    C = groups * width
    x, dy, w, b = make((20,), groups, width, act, seed=4)
    big = torch.full((20, C + 5), 3.0, dtype=x.dtype, device="cuda")
    view = big[:, 1:1 + C]
    view.copy_(x)
    y, mean, rstd = sm.layer_norm(view, w, b, groups=groups)
    check_norm(x, w, b, groups, 1e-5, y, mean, rstd)
    dx, dw, db = sm.layer_norm_backward(dy, x, w, mean, rstd, groups=groups)
    bigdy = torch.zeros(20, C + 3, dtype=x.dtype, device="cuda")
    bigdy[:, 3:].copy_(dy)
    got = sm.layer_norm_backward(bigdy[:, 3:], view, w, mean, rstd, groups=groups)
    check_gradients(x, dy, w, mean, rstd, groups, *got)
    sm.layer_norm(view, w, b, groups=groups, out=view)
    check_norm(x, w, b, groups, 1e-5, view, mean, rstd)
    assert bool((big[:, 0] == 3.0).all()) and bool((big[:, 1 + C:] == 3.0).all())


def test_values_far_from_zero():
    """A spread a thousandth of the offset: the variance is taken around the mean."""
    gen = torch.Generator().manual_seed(3)
    x = (1000.0 + torch.randn(17, 640, generator=gen)).cuda()
    w = torch.ones(640, device="cuda")
    check_norm(x, w, None, 1, 1e-5, *sm.layer_norm(x, w, None))


def check_gradients(x, dy, w, mean, rstd, groups, dx, dw, db):
    W = x.shape[-1] // groups
    rows = x.numel() // x.shape[-1]
    xd, gd = x.double().reshape(rows, groups, W), dy.double().reshape(rows, groups, W)
    m, r = mean.double().reshape(rows, groups, 1), rstd.double().reshape(rows, groups, 1)
    wd = torch.ones(1, groups, W, dtype=torch.float64, device="cuda") if w is None else w.double().view(1, groups, W)
    xh, dh = (xd - m) * r, gd * wd
    m1, m2 = dh.mean(-1, keepdim=True), (dh * xh).mean(-1, keepdim=True)
    ref = r * (dh - m1 - xh * m2)
    a1, a2 = dh.abs().mean(-1, keepdim=True), (dh * xh).abs().mean(-1, keepdim=True)
    # x - m loses 2^-24 of the larger of the two
    exh = U * (xd.abs() + m.abs()) * r + 2 * U * xh.abs()
    e = r * ((W + 8) * U * (a1 + xh.abs() * a2 + dh.abs()) + exh * a2 + xh.abs() * (dh.abs() * exh).mean(-1, keepdim=True)
             + 8 * U * (dh.abs() + a1 + xh.abs() * a2))
    e = e + torch.finfo(x.dtype).eps / 2 * (ref.abs() + e)
    got = dx.double().reshape(rows, groups, W)
    assert bool(((got - ref).abs() <= e).all()), float(((got - ref).abs() / e).max())
    ew = ((rows + 8) * U * (gd * xh).abs().sum(0) + (gd.abs() * exh).sum(0)).flatten()
    assert bool(((dw.double() - (gd * xh).sum(0).flatten()).abs() <= ew + 1e-30).all())
    assert bool(((db.double() - gd.sum(0).flatten()).abs() <= ((rows + 8) * U * gd.abs().sum(0)).flatten() + 1e-30).all())


@pytest.mark.parametrize("lead,groups,width", SHAPES)
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_backward(lead, groups, width, act):
    x, dy, w, b = make(lead, groups, width, act, seed=width + 1)
    _, mean, rstd = sm.layer_norm(x, w, b, groups=groups)
    check_gradients(x, dy, w, mean, rstd, groups, *sm.layer_norm_backward(dy, x, w, mean, rstd, groups=groups))
    check_gradients(x, dy, None, mean, rstd, groups, *sm.layer_norm_backward(dy, x, None, mean, rstd, groups=groups))


@pytest.mark.parametrize("offset", [1, 2, 4, 8])
@pytest.mark.parametrize("lead,groups,width", [((3,), 1, 2688), ((1300,), 1, 1024), ((7,), 4, 128), ((2,), 1, 16384)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_parameters_at_any_float(lead, groups, width, act, offset):
    """weight and bias as slices of longer vectors, from one float's alignment to a vector's."""
    x, dy, w, b = make(lead, groups, width, act, seed=offset)
    C = groups * width
    ws, bs = torch.zeros(C + 8, device="cuda"), torch.zeros(C + 8, device="cuda")
    ws[offset:offset + C], bs[offset:offset + C] = w, b
    w, b = ws[offset:offset + C], bs[offset:offset + C]
    y, mean, rstd = sm.layer_norm(x, w, b, groups=groups)
    check_norm(x, w, b, groups, 1e-5, y, mean, rstd)
    check_gradients(x, dy, w, mean, rstd, groups, *sm.layer_norm_backward(dy, x, w, mean, rstd, groups=groups))


def test_gradient_against_fp64_autograd_and_bits():
    x, dy, w, b = make((64,), 2, 96, "f32", seed=5)
    y, mean, rstd = sm.layer_norm(x, w, b, groups=2)
    leaves = [t.double().requires_grad_(True) for t in (x, w, b)]
    ref = torch.autograd.grad((norm64(*leaves, 2, 1e-5)[0] * dy.double()).sum(), leaves)
    got = sm.layer_norm_backward(dy, x, w, mean, rstd, groups=2)
    for g, r in zip(got, ref):        # 64 to 96 terms of a size around 1: 2^-24 x 100 terms x 16
        assert float((g.double() - r).abs().max()) <= 1e-4 * float(r.abs().max())
    again = sm.layer_norm_backward(dy, x, w, mean, rstd, groups=2)
    assert all(torch.equal(a, c) for a, c in zip(got, again))


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = sm.layer_norm(x, w, None, groups=2)
    assert y.shape == (0, 64) and mean.shape == (0, 2)
    dx, dw, db = sm.layer_norm_backward(x, x, w, mean, rstd, groups=2)
    assert dx.shape == (0, 64) and not bool(dw.any()) and not bool(db.any())


def test_nan_stays_in_its_group():
    x, _, w, b = make((6,), 3, 128, "bf16", seed=2)
    clean = sm.layer_norm(x, w, b, groups=3)[0]
    x[2, 130] = float("nan")
    y = sm.layer_norm(x, w, b, groups=3)[0]
    assert bool(y[2, 128:256].isnan().all())
    y[2, 128:256] = clean[2, 128:256]
    assert torch.equal(y, clean)


def test_captured():
    x, dy, w, b = make((128,), 1, 2688, "bf16", seed=8)

    def once():
        y, mean, rstd = sm.layer_norm(x, w, b)
        return [y, mean, rstd, *sm.layer_norm_backward(dy, x, w, mean, rstd)]

    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once()
    x.mul_(0.5).add_(0.25)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, once()))
