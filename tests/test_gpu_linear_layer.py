"""A layer's mixing made of the linear attention's and the layer norm's entry points, as a model would
run them (needs a B200): norm -> packed q|k|v projection -> linear attention on column slices -> norm per
head -> out projection -> residual, for a packed prompt on state slots and then token by token from a
captured graph; and the gradient of norm -> linear attention -> norm per head back to the layer's input.

Bounds, as relative 2-norms. bf16: q, k and v each carry two roundings (the norm's output and their own),
attention is linear in each of them (6), rounds scores and states (2) and its output (1); the norm per head
and the out projection round once each (2): eleven times the largest rounding, 2^-8. fp32: three links,
each with its values and its gradient, each within steps(d, L) roundings of 2^-24.
"""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import attention64, norm64, steps

pytestmark = pytest.mark.gpu


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


class Layer:
    """Weights of one layer and its two forms."""

    def __init__(self, D, H, G, dk, dv, seed):
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen) * std).cuda()

        self.D, self.H, self.G, self.dk, self.dv = D, H, G, dk, dv
        self.cols = (H * dk, G * dk, G * dv)
        self.w_in = normal(sum(self.cols), D, std=D ** -0.5).bfloat16()
        self.w_out = normal(D, H * dv, std=(H * dv) ** -0.5).bfloat16()
        self.n1, self.b1 = 1.0 + normal(D, std=0.1), normal(D, std=0.1)
        self.n2, self.b2 = 1.0 + normal(H * dv, std=0.1), normal(H * dv, std=0.1)
        self.log_decay = -(2.0 ** -torch.linspace(1, 7, H)).cuda()
        self.ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def dims(self, b, L):
        return sm.LinearDims(b, L, self.H, self.G, self.dk, self.dv, scale=self.dk ** -0.5, act="bf16")

    def run(self, h, attend):
        """h [T, D] bf16 through the layer; attend(q, k, v) is the call of the attention."""
        n = sm.layer_norm(h, self.n1, self.b1)[0]
        qkv = h.new_empty(h.shape[0], sum(self.cols))
        sm.ssd_mixer_projection(n, self.w_in, qkv, self.ws)
        o = attend(*qkv.split(self.cols, -1))
        o = sm.layer_norm(o, self.n2, self.b2, groups=self.H)[0]
        y = torch.empty_like(h)
        sm.ssd_mixer_projection(o, self.w_out, y, self.ws)
        return y

    def exact(self, h, init):
        """One sequence [L, D] in fp64: (y, final state)."""
        L = h.shape[0]
        n = norm64(h.double(), self.n1.double(), self.b1.double(), 1, 1e-5)[0]
        q, k, v = (n @ self.w_in.double().T).split(self.cols, -1)
        o, final = attention64(q.view(1, L, self.H, self.dk), k.view(1, L, self.G, self.dk), v.view(1, L, self.G, self.dv),
                               self.log_decay, init[None].double(), self.dk ** -0.5)
        o = norm64(o.reshape(L, -1), self.n2.double(), self.b2.double(), self.H, 1e-5)[0]
        return o @ self.w_out.double().T, final[0]


@pytest.mark.parametrize("H,G,dk,dv", [(4, 2, 64, 128), (3, 3, 32, 16)])
def test_prompts_then_tokens_from_a_graph(H, G, dk, dv):
    D, new, lens, slots = 320, 6, [1, 150, 0, 411, 7], [5, 0, 3, 2, 6]
    layer = Layer(D, H, G, dk, dv, seed=H)
    gen = torch.Generator().manual_seed(1)
    full = [torch.randn(n + new, D, generator=gen).bfloat16().cuda() for n in lens]
    init = torch.randn(8, H, dv, dk, generator=gen).cuda()
    has = [1, 0, 0, 1, 1]
    state = init.clone()
    state[slots[2]] = 0.0                      # a sequence that has no prompt yet starts from nothing
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    slot = torch.tensor(slots, dtype=torch.int32, device="cuda")
    flags = torch.tensor(has, dtype=torch.uint8, device="cuda")

    prompt = torch.cat([f[:n] for f, n in zip(full, lens)])
    y = layer.run(prompt, lambda q, k, v: sm.linear_prefill_varlen(layer.dims(len(lens), len(prompt)), cu, slot, flags,
                                                                   q, k, v, layer.log_decay, state))
    tokens = torch.stack([f[n:] for f, n in zip(full, lens)], 1)         # [new, b, D]
    h, out = torch.empty_like(tokens[0]), []

    def step():
        return layer.run(h, lambda q, k, v: sm.linear_decode_step(layer.dims(len(lens), 1), q, k, v, layer.log_decay,
                                                                  state, slot))
    h.copy_(tokens[0])
    out.append(step())
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for t in tokens[1:]:
        h.copy_(t)
        graph.replay()
        out.append(held.clone())
    out = torch.stack(out, 1)
    torch.cuda.synchronize()
    for i, n in enumerate(lens):
        ref, final = layer.exact(full[i], init[slots[i]] * has[i])
        got = torch.cat([y[cu[i]:cu[i + 1]], out[i]])
        assert rel(got, ref) <= 11 * 2.0 ** -8
        assert rel(state[slots[i]], final) <= 11 * 2.0 ** -8
    for s in set(range(8)) - set(slots):
        assert torch.equal(state[s], init[s])


@pytest.mark.parametrize("b,L,H,G,dk,dv", [(2, 90, 3, 3, 16, 32), (1, 200, 4, 2, 64, 64), (3, 1, 2, 1, 32, 16)])
def test_gradient_through_norms_and_attention(b, L, H, G, dk, dv):
    cols = (H * dk, G * dk, G * dv)
    gen = torch.Generator().manual_seed(L)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).cuda()

    x, dy = normal(b, L, sum(cols)), normal(b, L, H * dv)
    n1, b1, n2, b2 = 1 + 0.1 * normal(sum(cols)), 0.1 * normal(sum(cols)), 1 + 0.1 * normal(H * dv), 0.1 * normal(H * dv)
    g = -(2.0 ** -torch.linspace(1, 6, H)).cuda()
    d = sm.LinearDims(b, L, H, G, dk, dv, scale=dk ** -0.5, act="f32")

    n, m1, r1 = sm.layer_norm(x, n1, b1)
    q, k, v = n.split(cols, -1)
    o, _ = sm.linear_prefill(d, q, k, v, g)
    y, m2, r2 = sm.layer_norm(o, n2, b2, groups=H)
    do, dn2, db2 = sm.layer_norm_backward(dy, o, n2, m2, r2, groups=H)
    ga = sm.linear_backward(d, q, k, v, g, do)
    dx, dn1, db1 = sm.layer_norm_backward(torch.cat([ga["q"], ga["k"], ga["v"]], -1), x, n1, m1, r1)

    def chain(x, n1, b1, n2, b2):
        n = norm64(x, n1, b1, 1, 1e-5)[0]
        q, k, v = (t.view(b, L, h, -1) for t, h in zip(n.split(cols, -1), (H, G, G)))
        o, _ = attention64(q, k, v, g, None, dk ** -0.5)
        return norm64(o.reshape(b, L, -1), n2, b2, H, 1e-5)[0]

    leaves = [t.double().requires_grad_(True) for t in (x, n1, b1, n2, b2)]
    ref = chain(*leaves)
    grads = torch.autograd.grad((ref * dy.double()).sum(), leaves)
    tol = 6 * steps(d, L) * 2.0 ** -24
    assert rel(y, ref.detach()) <= tol
    for got, want in zip((dx, dn1, db1, dn2, db2), grads):
        assert rel(got, want) <= tol
    # and against differences of the fp64 chain, in one direction of all five: h^2 of a third derivative
    step = [torch.randn(t.shape, generator=gen).double().cuda() for t in (x, n1, b1, n2, b2)]
    h = 1e-5
    with torch.no_grad():
        up, down = (chain(*[t + s * h * e for t, e in zip(leaves, step)]) for s in (1, -1))
        slope = float(((up - down) * dy.double()).sum() / (2 * h))
    got = sum(float((a.double() * e).sum()) for a, e in zip((dx, dn1, db1, dn2, db2), step))
    size = sum(float(a.double().norm() * e.norm()) for a, e in zip((dx, dn1, db1, dn2, db2), step))
    assert abs(got - slope) <= (tol + 1e-6) * size
