"""Plain fp64 forms of linear attention with a decay per head and of the grouped layer norm, and the
error bounds that the GPU tests hold the kernels to.

The bounds are elementwise and follow from the arithmetic. Let A be the same sum with every factor
replaced by its absolute value (what the roundings of the terms scale with).
  * fp32: every term of a state or an output passes through at most `steps` roundings of 2^-24
    (one or two a token while it stays in the state, then the sum over dk lanes), so the error is at
    most steps * 2^-24 * A.
  * bf16 on the tensor cores: each score and each state operand is rounded once to bf16 (2^-8 of the
    term), so 2^-8 A, plus the result's own rounding, 2^-8 |o|, plus the fp32 part. States are added
    to from sums of three bf16, each half a step (2^-8) of what the ones before leave: 2^-24 A plus
    the fp32 part.
"""
from __future__ import annotations

import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attention64(q, k, v, log_decay, init, scale):
    """q [b, L, H, dk], k [b, L, G, dk], v [b, L, G, dv], init [b, H, dv, dk] or None, all fp64:
    (o [b, L, H, dv], final state)."""
    b, L, H, _ = q.shape
    r = H // k.shape[2]
    k, v = k.repeat_interleave(r, dim=2), v.repeat_interleave(r, dim=2)
    g = log_decay.double().clamp(min=-1e4)
    t = torch.arange(L, device=q.device, dtype=torch.float64)
    gap = t[:, None] - t[None, :]
    w = torch.exp(g[:, None, None] * gap.clamp(min=0)) * (gap >= 0)
    s = torch.einsum("bthe,bjhe->bhtj", q, k) * w
    o = torch.einsum("bhtj,bjhd->bthd", s, v)
    left = torch.exp(g[:, None] * (L - 1 - t)) if L else torch.zeros(H, 0, dtype=torch.float64, device=q.device)
    final = torch.einsum("bjhd,hj,bjhe->bhde", v, left, k)
    if init is not None:
        o = o + torch.einsum("ht,bthe,bhde->bthd", torch.exp(g[:, None] * (t + 1)), q, init)
        final = final + torch.exp(g * L)[None, :, None, None] * init
    return scale * o, final


def make(b, L, H, G, dk, dv, act, seed, init=True, device="cuda", decay=None):
    """Seeded inputs: q, k, v (packed row layout), log_decay and an initial state."""
    gen = torch.Generator(device="cpu").manual_seed(seed)
    a = torch.bfloat16 if act == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    x = {"q": normal(b, L, H * dk), "k": normal(b, L, G * dk), "v": normal(b, L, G * dv), "do": normal(b, L, H * dv)}
    x = {n: t.to(a).to(device) for n, t in x.items()}
    slope = -(2.0 ** (-8.0 * torch.rand(H, generator=gen)))
    x["log_decay"] = (slope if decay is None else torch.tensor(decay, dtype=torch.float32).repeat(H)[:H]).to(device)
    x["init"] = normal(b, H, dv, dk).to(device) if init else None
    x["dfinal"] = normal(b, H, dv, dk).to(device) if init else None
    return x


def dims(b, L, H, G, dk, dv, act, scale=None):
    return sm.LinearDims(b, L, H, G, dk, dv, scale=dk ** -0.5 if scale is None else scale, act=act)


def wide(x, d):
    """The fp64 operands of attention64."""
    b, L = x["q"].shape[0], x["q"].shape[1]
    return (x["q"].double().view(b, L, d.nheads, d.dk), x["k"].double().view(b, L, d.ngroups, d.dk),
            x["v"].double().view(b, L, d.ngroups, d.dv))


def steps(d, L):
    """Roundings a term meets at most in fp32: three a token (or, chunk by chunk, fewer), the lanes'
    sum, the decay factors."""
    return 3 * L + d.dk + d.dv + 16


def check(name, got, ref, mag, d, L, state=False):
    """|got - ref| within the bound above, mag being A."""
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    tol = steps(d, L) * 2.0 ** -24 * mag
    if d.act == "bf16":
        tol = tol + (2.0 ** -24 * mag if state else 2.0 ** -8 * (mag + ref.abs()))
    bad = ~((got - ref).abs() <= tol + 1e-30)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst "
                                 f"{float(((got - ref).abs() / (tol + 1e-30)).nan_to_num(nan=float('inf')).max()):.3g} x the bound")


def gradients64(q, k, v, log_decay, init, scale, do, dfinal):
    """fp64 gradients by differentiating attention64: dict like linear_backward's."""
    leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
    i = (torch.zeros(q.shape[0], q.shape[2], v.shape[3], q.shape[3], dtype=torch.float64, device=q.device)
         if init is None else init.detach().clone()).requires_grad_(True)
    o, final = attention64(*leaves, log_decay, i, scale)
    loss = (o * do).sum() + ((final * dfinal).sum() if dfinal is not None else 0.0)
    g = torch.autograd.grad(loss, [*leaves, i])
    return dict(zip(("q", "k", "v", "init_state"), g))


def norm64(x, weight, bias, groups, eps):
    """fp64 grouped layer norm: (y, mean, rstd)."""
    h = x.unflatten(-1, (groups, x.shape[-1] // groups))
    mean = h.mean(-1)
    c = h - mean[..., None]
    rstd = 1.0 / torch.sqrt((c * c).mean(-1) + eps)
    y = (c * rstd[..., None]).flatten(-2)
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd
