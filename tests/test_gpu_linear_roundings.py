"""What the scans on tensor cores round (needs a B200): outputs and gradients in bf16 are the fp32 arithmetic's, rounded once.

Inputs are one-hot over a few features, so that a score is one product of two bf16 numbers (16 bits, exact in
fp32), each of its factors and sums is known to be few, and A of tests/linear_util.py (the sums over absolute
values) is close to the results themselves. Of an output then
  * scores and state operands are sums of two bf16: half a step of what the first leaves, 2^-8 * 2^-8 = 2^-16 A;
  * the fp32 arithmetic takes at most steps(d, L) roundings, steps 2^-24 A.
With delta their sum, x the value and y what the kernel rounds (|y - x| <= delta), rounding to nearest gives
|fl(y) - x| <= |fl(y) - y| + delta <= |fl(x) - y| + delta <= |fl(x) - x| + 2 delta."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import attention64, dims, gradients64, make, steps, wide

pytestmark = pytest.mark.gpu


def one_hot(x, n, d, gen, features=8):
    """x [b, L, n * d] with all but one of `features` columns of each head zeroed, another column for each token."""
    b, L, _ = x.shape
    cols = torch.randperm(d, generator=gen)[:features]
    at = cols[torch.randint(features, (b, L, n, 1), generator=gen)].to(x.device)
    x = x.view(b, L, n, d)
    return torch.zeros_like(x).scatter(3, at, x.gather(3, at)).view(b, L, n * d)


def sparse(shape, seed, init):
    b, L, H, G, dk, dv = shape
    x = make(*shape, "bf16", seed=seed, init=init)
    gen = torch.Generator().manual_seed(seed)
    for name, n, d in (("q", H, dk), ("k", G, dk), ("v", G, dv), ("do", H, dv)):
        x[name] = one_hot(x[name], n, d, gen)
    return x


def check_rounded_once(name, got, ref, mag, d, L):
    delta = (2.0 ** -16 + steps(d, L) * 2.0 ** -24) * mag
    own = (ref.to(torch.bfloat16).double() - ref).abs()
    bad = ~((got.double() - ref).abs() <= own + 2 * delta + 1e-30)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} values are off by more than one rounding"


# heads of each pair of dims, several blocks and a ragged end, a row in one piece and one in several
@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("shape", [(2, 300, 3, 3, 64, 64), (1, 389, 2, 2, 64, 128), (2, 257, 2, 1, 128, 64), (2, 300, 4, 2, 128, 128),
                                   (1, 1500, 2, 2, 128, 128)])
def test_results_are_rounded_once(shape, init):
    b, L, H, G, dk, dv = shape
    d = dims(*shape, "bf16")
    x = sparse(shape, sum(shape), init)
    i, df = (None if x[n] is None else x[n].double() for n in ("init", "dfinal"))
    q, k, v = wide(x, d)
    do = x["do"].double().view(b, L, H, dv)

    def size(t):
        return None if t is None else t.abs()

    o, _ = sm.linear_prefill(d, x["q"], x["k"], x["v"], x["log_decay"], x["init"])
    ref, _ = attention64(q, k, v, x["log_decay"], i, d.scale)
    mag, _ = attention64(size(q), size(k), size(v), x["log_decay"], size(i), d.scale)
    check_rounded_once("o", o.view(ref.shape), ref, mag, d, L)

    g = sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"])
    ref = gradients64(q, k, v, x["log_decay"], i, d.scale, do, df)
    mag = gradients64(size(q), size(k), size(v), x["log_decay"], size(i), d.scale, size(do), size(df))
    for n in ("q", "k", "v"):
        check_rounded_once("d" + n, g[n].view(ref[n].shape), ref[n], mag[n], d, L)
