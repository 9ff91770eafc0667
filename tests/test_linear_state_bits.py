"""The precision that linear attention's states promise: products of 24-bit operands, decays that are not rounded to
fp32 in every step. The GPU tests need a B200; the CPU tests show that their bounds tell the promised arithmetic
from the next cheaper one.

One token (u = 2^-24). Where all but one token's v are zero, the state is w v k^T, w = l^e. The power is within 8 u
(expf 4 u, its correction, the products); w v takes one rounding more, its three bf16 terms leave at most u, and each
of their products with k (exact) is added in fp32, 2 u each if sums are cut off and not rounded: 8 + 1 + 1 + 6 = 16 u,
and |g| e u for the exponent. Two terms leave up to 2^-16 = 256 u, 2^-18 = 64 u or more in half of all values.

A slow decay (l = 1 - 1.1e-5, 16384 tokens of positive v and k, S positive). Token by token each step rounds three
times, each time by at most u of S and as often up as down: 8 sqrt(3 L) u (eight standard deviations at the very
least). On tensor cores only every 128th token does, beside the block's own sums, 24 additions of at most 2 u each and
the 16 u above. l rounded to fp32 is off by 2^-25 (this l is one of the worst), for L / 2 steps on average."""
import math

import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import dims

U = 2.0 ** -24
DECAYS = [-0.013, -0.3, -1.7]
SLOW = -1.0937499610008672e-05


def one_token(dk, dv, seed, L=300, at=262):
    """bf16 k and v of token `at` (of three blocks of 128, the last one short), heads of different decays."""
    gen = torch.Generator().manual_seed(seed)
    H = len(DECAYS)
    k, v = torch.randn(1, L, H, dk, generator=gen).bfloat16(), torch.zeros(1, L, H, dv).bfloat16()
    v[:, at] = torch.randn(1, H, dv, generator=gen).bfloat16()
    return k, v, torch.tensor(DECAYS, dtype=torch.float32)


def one_token_bound(g, e):
    return (16 + g.double().abs() * e) * U


def off(state, ref, bound):
    """The largest error of [H, dv, dk] states relative to the bound of their head."""
    return float(((state.double() - ref).abs() / (bound.view(-1, 1, 1) * ref.abs() + 1e-300)).max())


def outer(w, v, k):
    return w.view(-1, 1, 1) * v[..., None] * k[:, None]


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_state_keeps_24_bits(dk, dv):
    """The state after the row, and the gradient of the one before it (the reverse scan, with do in v's place)."""
    L, at, H = 300, 262, len(DECAYS)
    k, v, g = one_token(dk, dv, seed=dk + dv, L=L, at=at)
    d = dims(1, L, H, H, dk, dv, "bf16", scale=1.0)
    rows = [t.reshape(1, L, -1).cuda() for t in (k, v)]
    q = torch.zeros_like(rows[0])
    _, state = sm.linear_prefill(d, q, *rows, g.cuda())
    e = L - 1 - at
    ref = outer(torch.exp(g.double() * e), v[0, at].double(), k[0, at].double())
    assert off(state[0].cpu(), ref, one_token_bound(g, e)) <= 1

    mirror = [t.flip(1).contiguous() for t in rows]                      # the token at L - 1 - at
    none = torch.zeros_like(mirror[1])
    grad = sm.linear_backward(d, mirror[0], torch.zeros_like(mirror[0]), none, g.cuda(), mirror[1])["init_state"]
    ref = outer(torch.exp(g.double() * (e + 1)), v[0, at].double(), k[0, at].double())
    assert off(grad[0].cpu(), ref, one_token_bound(g, e + 1)) <= 1


def test_two_terms_would_not_keep_them():
    for dk, dv in [(64, 64), (128, 128)]:
        k, v, g = one_token(dk, dv, seed=dk + dv)
        e, at = 37, 262
        w = torch.exp(g.double() * e)
        t = w.float()[:, None] * v[0, at].float()
        ref = outer(w, v[0, at].double(), k[0, at].double())
        terms, left = [], t
        for _ in range(3):
            terms.append(left.bfloat16().float())
            left = left - terms[-1]
        kk = k[0, at].double()[:, None]
        two, three = ((sum(x.double() for x in terms[:n]))[..., None] * kk for n in (2, 3))
        assert off(two, ref, one_token_bound(g, e)) > 2
        assert off(three, ref, one_token_bound(g, e)) <= 1


def slow_row(L, H, dk, dv, act, seed):
    gen = torch.Generator().manual_seed(seed)
    a = torch.bfloat16 if act == "bf16" else torch.float32
    k, v = ((0.5 + torch.rand(1, L, H, n, generator=gen)).to(a) for n in (dk, dv))
    return k, v, torch.full((H,), SLOW)


def slow_state(k, v, lam):
    L = k.shape[1]
    w = torch.exp(math.log(lam) * torch.arange(L - 1, -1, -1, dtype=torch.float64))
    return torch.einsum("t,thd,the->hde", w, v[0].double(), k[0].double())


def slow_bound(act, L):
    return (8 * math.sqrt(3 * L) if act == "f32" else 48 + 16 + 8 * math.sqrt(3 * L / 128)) * U


@pytest.mark.gpu
@pytest.mark.parametrize("act,dk,dv", [("f32", 16, 16), ("f32", 64, 32), ("bf16", 64, 64), ("bf16", 128, 128)])
def test_a_slow_decay_is_not_rounded(act, dk, dv):
    L, H = 16384, 2
    k, v, g = slow_row(L, H, dk, dv, act, seed=dk)
    d = dims(1, L, H, H, dk, dv, act)
    rows = [t.reshape(1, L, -1).cuda() for t in (k, v)]
    _, state = sm.linear_prefill(d, torch.zeros_like(rows[0]), *rows, g.cuda())
    ref = slow_state(k, v, math.exp(float(g[0])))
    assert off(state[0].cpu(), ref, torch.full((H,), slow_bound(act, L), dtype=torch.float64)) <= 1


def test_a_rounded_decay_would_be_seen():
    L, H = 16384, 2
    k, v, g = slow_row(L, H, 16, 16, "f32", seed=16)
    lam = math.exp(float(g[0]))
    rounded = float(torch.tensor(lam, dtype=torch.float32))
    assert abs(rounded - lam) > 0.99 * 2.0 ** -25
    ref = slow_state(k, v, lam)
    assert off(slow_state(k, v, rounded), ref, torch.full((H,), slow_bound("f32", L), dtype=torch.float64)) > 2
