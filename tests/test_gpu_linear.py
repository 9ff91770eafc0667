"""GPU parity of linear attention with a decay per head (prefill, packed prefill, decode, backward)
with its fp64 form (needs a B200). Bounds: tests/linear_util.py."""
import math

import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import attention64, check, dims, gradients64, make, wide

pytestmark = pytest.mark.gpu

# (b, L, H, G, dk, dv): one token, a block's edges, several blocks, shared heads, uneven head counts
SHAPES = [
    (1, 1, 1, 1, 64, 64), (2, 2, 3, 1, 64, 128), (1, 127, 2, 2, 128, 64), (1, 128, 4, 2, 128, 128),
    (3, 129, 2, 1, 64, 64), (2, 257, 5, 5, 128, 128), (1, 700, 3, 3, 64, 128), (1, 1100, 2, 1, 128, 128),
    (2, 300, 300, 300, 64, 64), (2, 7, 3, 3, 128, 64), (1, 8, 2, 1, 64, 64), (3, 9, 2, 2, 128, 128),
]
SMALL = [(2, 37, 3, 3, 16, 32), (1, 200, 4, 2, 32, 16), (1, 65, 2, 2, 16, 16), (2, 190, 6, 2, 128, 32), (1, 333, 2, 1, 64, 16)]
ALL = [(s, a) for s in SHAPES for a in ("bf16", "f32")] + [(s, a) for s in SMALL for a in ("bf16", "f32")]


def forward(x, d, **kw):
    return sm.linear_prefill(d, x["q"], x["k"], x["v"], x["log_decay"], x["init"], **kw)


def check_forward(x, d, o, fs, scale):
    q, k, v = wide(x, d)
    i = None if x["init"] is None else x["init"].double()
    ref, rf = attention64(q, k, v, x["log_decay"], i, scale)
    mag, mf = attention64(q.abs(), k.abs(), v.abs(), x["log_decay"], None if i is None else i.abs(), abs(scale))
    L = q.shape[1]
    check("o", o.view(ref.shape), ref, mag, d, L)
    check("final_state", fs, rf, mf, d, L, state=True)


@pytest.mark.parametrize("shape,act", ALL)
@pytest.mark.parametrize("init", [True, False])
def test_prefill(shape, act, init):
    d = dims(*shape, act)
    x = make(*shape, act, seed=sum(shape), init=init)
    check_forward(x, d, *forward(x, d), d.scale)


@pytest.mark.parametrize("decay", [[0.0], [-math.inf], [-1e-6, -30.0], [-0.7, 0.0, -200.0]])
@pytest.mark.parametrize("act,shape", [("bf16", (1, 300, 3, 3, 64, 64)), ("f32", (1, 300, 3, 3, 32, 16))])
def test_extreme_decays(decay, act, shape):
    d = dims(*shape, act)
    x = make(*shape, act, seed=7, decay=decay)
    check_forward(x, d, *forward(x, d), d.scale)


@pytest.mark.parametrize("act,shape", [("bf16", (2, 150, 2, 2, 64, 128)), ("f32", (2, 50, 2, 2, 16, 16))])
def test_column_slices_of_one_row(act, shape):
    """q, k, v and o as column slices of packed rows, with gaps between the rows."""
    b, L, H, G, dk, dv = shape
    d = dims(*shape, act, scale=-0.3)
    x = make(*shape, act, seed=3)
    pad = 16
    packed = torch.full((b, L, H * dk + G * (dk + dv) + pad), float("nan"), dtype=d.torch_dtype, device="cuda")
    at = 0
    y = dict(x)
    for n in ("k", "q", "v"):
        w = x[n].shape[-1]
        packed[..., at:at + w] = x[n]
        y[n] = packed[..., at:at + w]
        at += w
    wideo = torch.zeros(b, L, H * dv + pad, dtype=d.torch_dtype, device="cuda")
    fs = torch.empty_like(x["init"])
    o, fs = forward(y, d, out=(wideo[..., :H * dv], fs))
    check_forward(x, d, o.contiguous(), fs, d.scale)
    assert not bool(wideo[..., H * dv:].any())


@pytest.mark.parametrize("act,shape", [("bf16", (1, 1500, 2, 2, 128, 64)), ("f32", (1, 900, 2, 1, 32, 64)), ("bf16", (2, 0, 2, 2, 64, 64))])
def test_state_in_place_and_pieces(act, shape):
    """A row in two calls chained through the states equals one call's bound; the final state may be
    the initial one's buffer; L = 0 hands the state on."""
    b, L, H, G, dk, dv = shape
    d = dims(*shape, act)
    x = make(*shape, act, seed=11)
    st = x["init"].clone()
    cut = L * 2 // 5
    os = []
    for t0, t1 in ((0, cut), (cut, L)):
        dd = dims(b, t1 - t0, H, G, dk, dv, act)
        y = {n: x[n][:, t0:t1].contiguous() for n in ("q", "k", "v")}
        o = torch.empty(b, t1 - t0, H * dv, dtype=d.torch_dtype, device="cuda")
        sm.linear_prefill(dd, y["q"], y["k"], y["v"], x["log_decay"], st, out=(o, st))
        os.append(o)
    check_forward(x, d, torch.cat(os, 1), st, d.scale)


LENS = [[1], [0], [5, 0, 1, 130], [128, 256, 1, 127], [900, 3], [0, 0, 1000, 0], [64] * 20, [1] * 33, [7, 8, 9, 10, 0, 300, 8],
        [1] * 40 + [2500, 2]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:5])))
@pytest.mark.parametrize("act,H,G,dk,dv", [("bf16", 4, 2, 64, 128), ("f32", 2, 2, 32, 16), ("bf16", 2, 1, 32, 32),
                                           ("bf16", 40, 40, 128, 128)])
def test_packed(lens, act, H, G, dk, dv):
    """Packed sequences on slots: rows behind the last one, slots that no sequence owns and the other
    sequences' NaN stay out."""
    b, T = len(lens), sum(lens) + 9
    d = dims(b, T, H, G, dk, dv, act)
    x = make(1, T, H, G, dk, dv, act, seed=T)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    nslots = b + 2
    gen = torch.Generator().manual_seed(b)
    slots = torch.randperm(nslots, generator=gen)[:b]
    has = torch.arange(b) % 3 != 1
    state = torch.randn(nslots, H, dv, dk, generator=gen).cuda()
    bad = max(range(b), key=lambda i: lens[i]) if b > 1 else None      # a sequence of NaN
    q, k, v = (x[n][0].clone() for n in ("q", "k", "v"))
    if bad is not None:
        k[cu[bad]:cu[bad + 1]] = float("nan")
        v[cu[bad]:cu[bad + 1]] = float("nan")
    k[cu[-1]:], v[cu[-1]:] = float("nan"), float("inf")
    before = state.clone()
    o = torch.full((T, H * dv), 7.0, dtype=d.torch_dtype, device="cuda")
    sm.linear_prefill_varlen(d, cu.cuda(), slots.to(torch.int32).cuda(), has.to(torch.uint8).cuda(), q, k, v, x["log_decay"],
                             state, o=o)
    assert bool((o[cu[-1]:] == 7.0).all())
    free = [s for s in range(nslots) if s not in slots.tolist()]
    assert torch.equal(state[free], before[free])
    for i in range(b):
        if i == bad:
            continue
        n = lens[i]
        y = {m: x[m][:, cu[i]:cu[i + 1]] for m in ("q", "k", "v")}
        y |= {"log_decay": x["log_decay"], "init": before[slots[i]][None] if has[i] else None}
        check_forward(y, dims(1, n, H, G, dk, dv, act), o[cu[i]:cu[i + 1]][None], state[slots[i]][None], d.scale)


def test_packed_skips_slots_out_of_range():
    H, dk, dv, lens = 2, 64, 64, [40, 200, 7]
    T = sum(lens)
    d = dims(3, T, H, H, dk, dv, "bf16")
    x = make(1, T, H, H, dk, dv, "bf16", seed=1)
    cu = torch.tensor([0, 40, 240, 247], dtype=torch.int32, device="cuda")
    state = torch.randn(4, H, dv, dk, device="cuda")
    before = state.clone()
    o = torch.full((T, H * dv), 7.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([-1, 2, 4], dtype=torch.int32, device="cuda")
    sm.linear_prefill_varlen(d, cu, slots, None, x["q"][0], x["k"][0], x["v"][0], x["log_decay"], state, o=o)
    assert bool((o[:40] == 7.0).all()) and bool((o[240:] == 7.0).all())
    assert torch.equal(state[[0, 1, 3]], before[[0, 1, 3]])
    y = {m: x[m][:, 40:240] for m in ("q", "k", "v")} | {"log_decay": x["log_decay"], "init": before[2][None]}
    check_forward(y, dims(1, 200, H, H, dk, dv, "bf16"), o[40:240][None], state[2][None], d.scale)


DECODE = [(1, 1, 1, 16, 16), (3, 5, 5, 64, 64), (2, 8, 2, 128, 128), (33, 4, 1, 32, 128), (5, 6, 3, 128, 16), (300, 2, 2, 64, 32)]


@pytest.mark.parametrize("b,H,G,dk,dv", DECODE)
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_decode_on_slots(b, H, G, dk, dv, act):
    d = dims(b, 1, H, G, dk, dv, act)
    x = make(b, 1, H, G, dk, dv, act, seed=b + dk)
    nslots = b + 3
    gen = torch.Generator().manual_seed(5)
    slots = torch.randperm(nslots, generator=gen)[:b].to(torch.int32)
    skipped = 0 if b > 1 else None
    if skipped is not None:
        slots[skipped] = -1
    state = torch.randn(nslots, H, dv, dk, generator=gen).cuda()
    before = state.clone()
    o = torch.full((b, H * dv), 7.0, dtype=d.torch_dtype, device="cuda")
    sm.linear_decode_step(d, x["q"], x["k"], x["v"], x["log_decay"], state, slots.cuda(), o=o)
    used = [i for i in range(b) if i != skipped]
    y = {n: x[n][used] for n in ("q", "k", "v")} | {"log_decay": x["log_decay"], "init": before[slots[used].long()]}
    # fp32 arithmetic in every type: the result's rounding and a few of fp32
    q, k, v = wide(y, d)
    ref, rf = attention64(q, k, v, y["log_decay"], y["init"].double(), d.scale)
    mag, mf = attention64(q.abs(), k.abs(), v.abs(), y["log_decay"], y["init"].double().abs(), d.scale)
    half = torch.finfo(d.torch_dtype).eps / 2
    assert bool(((o[used].double() - ref.view(len(used), -1)).abs() <= half * ref.abs().view(len(used), -1)
                 + (dk + 8) * 2.0 ** -24 * mag.view(len(used), -1)).all())
    assert bool(((state[slots[used].long()].double() - rf).abs() <= 4 * 2.0 ** -24 * mf).all())
    rest = [s for s in range(nslots) if s not in slots[used].tolist()]
    assert torch.equal(state[rest], before[rest])
    if skipped is not None:
        assert bool((o[skipped] == 7.0).all())


def test_decode_continues_a_prefill():
    """Prefill of 200 tokens and 20 decode steps against one row of 220."""
    shape = (2, 220, 3, 3, 64, 128)
    d = dims(*shape, "bf16")
    x = make(*shape, "bf16", seed=21)
    y = {n: x[n][:, :200].contiguous() for n in ("q", "k", "v")} | {"log_decay": x["log_decay"], "init": x["init"]}
    o, st = forward(y, dims(2, 200, 3, 3, 64, 128, "bf16"))
    os = [o]
    dd = dims(2, 1, 3, 3, 64, 128, "bf16")
    for t in range(200, 220):
        os.append(sm.linear_decode_step(dd, x["q"][:, t], x["k"][:, t], x["v"][:, t], x["log_decay"], st)[:, None])
    check_forward(x, d, torch.cat(os, 1), st, d.scale)


@pytest.mark.parametrize("shape,act", ALL)
@pytest.mark.parametrize("init", [True, False])
def test_backward(shape, act, init):
    d = dims(*shape, act)
    x = make(*shape, act, seed=1 + sum(shape), init=init)
    g = sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"])
    check_backward(x, d, g)


def check_backward(x, d, g):
    q, k, v = wide(x, d)
    b, L = q.shape[:2]
    do = x["do"].double().view(b, L, d.nheads, d.dv)
    i, df = (None if x[n] is None else x[n].double() for n in ("init", "dfinal"))
    ref = gradients64(q, k, v, x["log_decay"], i, d.scale, do, df)
    mag = gradients64(q.abs(), k.abs(), v.abs(), x["log_decay"], None if i is None else i.abs(), abs(d.scale), do.abs(),
                      None if df is None else df.abs())
    for n in ("q", "k", "v"):
        check("d" + n, g[n].view(ref[n].shape), ref[n], mag[n], d, L)
    check("dinit_state", g["init_state"], ref["init_state"], mag["init_state"], d, L, state=True)


@pytest.mark.parametrize("act,dk,dv", [("bf16", 64, 128), ("f32", 16, 32)])
def test_backward_of_no_tokens(act, dk, dv):
    d = dims(2, 0, 3, 3, dk, dv, act)
    x = make(2, 0, 3, 3, dk, dv, act, seed=1)
    g = sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"])
    assert torch.equal(g["init_state"], x["dfinal"]) and g["q"].shape == (2, 0, 3 * dk)


@pytest.mark.parametrize("shape", [(1, 16384, 5, 5, 64, 64), (1, 6000, 2, 1, 128, 128), (5, 1290, 64, 64, 64, 64),
                                   (1, 2500, 20, 20, 128, 64), (1, 5001, 60, 60, 64, 64)])
def test_long_and_many_rows(shape):
    """Rows of many blocks, cut and whole, and more segments than SMs, forwards and backwards. The fp64
    form runs head by head; the bound is that of the sizes."""
    b, L, H, G, dk, dv = shape
    d = dims(*shape, "bf16")
    x = make(*shape, "bf16", seed=L)
    o, fs = forward(x, d)
    g = sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"]) if G == H else None
    one = dims(1, L, 1, 1, dk, dv, "bf16")
    for i, h in {(0, 0), (b - 1, H - 1), (b // 2, H // 2)}:
        r = H // G
        y = {"q": x["q"].view(b, L, H, dk)[i:i + 1, :, h], "do": x["do"].view(b, L, H, dv)[i:i + 1, :, h],
             "k": x["k"].view(b, L, G, dk)[i:i + 1, :, h // r], "v": x["v"].view(b, L, G, dv)[i:i + 1, :, h // r],
             "log_decay": x["log_decay"][h:h + 1], "init": x["init"][i:i + 1, h:h + 1], "dfinal": x["dfinal"][i:i + 1, h:h + 1]}
        check_forward(y, one, o.view(b, L, H, dv)[i:i + 1, :, h], fs[i:i + 1, h:h + 1], d.scale)
        if g is not None and L <= 6000:
            check_backward(y, one, {"q": g["q"].view(b, L, H, dk)[i:i + 1, :, h], "k": g["k"].view(b, L, G, dk)[i:i + 1, :, h],
                                    "v": g["v"].view(b, L, G, dv)[i:i + 1, :, h], "init_state": g["init_state"][i:i + 1, h:h + 1]})


@pytest.mark.parametrize("decay", [[0.0], [-math.inf], [-200.0, -1e-5]])
@pytest.mark.parametrize("act,shape", [("bf16", (1, 290, 2, 2, 128, 64)), ("f32", (1, 100, 2, 1, 16, 32))])
def test_backward_extreme_decays(decay, act, shape):
    d = dims(*shape, act)
    x = make(*shape, act, seed=9, decay=decay)
    check_backward(x, d, sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"]))


def test_gradient_against_differences():
    """<gradient, direction> against central differences of the fp32 forward call. A loss of n = 2.6e3
    products of size about 1 is off by less than n 2^-24 steps, about 1e-2 after division by 2h = 0.1
    at the most and far less on average; the third derivative is zero (the loss is a polynomial of
    degree one in each of q, k, v and the state)."""
    shape = (1, 40, 2, 1, 32, 32)
    d = dims(*shape, "f32")
    x = make(*shape, "f32", seed=2)
    g = sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"])

    def loss(y):
        o, fs = forward(y, d)
        return float((o.double() * x["do"].double()).sum() + (fs.double() * x["dfinal"].double()).sum())

    for n, key in (("q", "q"), ("k", "k"), ("v", "v"), ("init", "init_state")):
        u = torch.randn(x[n].shape, generator=torch.Generator().manual_seed(4)).cuda()
        h = 0.05
        diff = (loss(x | {n: x[n] + h * u}) - loss(x | {n: x[n] - h * u})) / (2 * h)
        want = float((g[key].double() * u.double()).sum())
        assert abs(diff - want) <= 1e-2 + 1e-4 * abs(want), (n, diff, want)


def test_captured_and_replayed():
    """One graph of a prefill, a decode step and a backward pass with their own workspaces, replayed on
    new inputs, gives what the plain calls give; two graphs do not share what they keep."""
    shape = (1, 400, 2, 1, 64, 64)
    d, dd = dims(*shape, "bf16"), dims(1, 1, 2, 1, 64, 64, "bf16")
    a, b = make(*shape, "bf16", seed=1), make(*shape, "bf16", seed=2)
    live = {n: t.clone() for n, t in a.items()}

    def once(y):
        o, st = forward(y, d)
        state = st.clone()
        step = sm.linear_decode_step(dd, y["q"][:, 0], y["k"][:, 0], y["v"][:, 0], y["log_decay"], state)
        g = sm.linear_backward(d, y["q"], y["k"], y["v"], y["log_decay"], y["do"], y["init"], y["dfinal"])
        return [o, st, step, state, *g.values()]

    once(live)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, once(live)))
    for n in live:
        live[n].copy_(b[n])
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = once(b)
    for _, got in graphs:
        for p, w in zip(got, want):
            assert torch.equal(p, w)


def test_another_stream():
    """Inputs made on the current stream, the call on another one that waits for it."""
    shape = (2, 500, 2, 2, 64, 64)
    d = dims(*shape, "bf16")
    x = make(*shape, "bf16", seed=8)
    want = forward(x, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = forward(x, d, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_same_inputs_same_bits():
    shape = (2, 1000, 4, 2, 128, 64)
    d = dims(*shape, "bf16")
    x = make(*shape, "bf16", seed=8)
    a, b = (forward(x, d) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = (sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"]) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("act,shape", [("bf16", (2, 300, 2, 2, 64, 64)), ("f32", (2, 40, 2, 2, 32, 32))])
def test_nan_stays_in_its_row_and_its_future(act, shape):
    """A NaN in one row's k at token t: the other row and the tokens before t are as without it."""
    d = dims(*shape, act)
    x = make(*shape, act, seed=6)
    clean, _ = forward(x, d)
    t = shape[1] * 2 // 3
    y = dict(x, k=x["k"].clone())
    y["k"][0, t] = float("nan")
    o, fs = forward(y, d)
    assert torch.equal(o[1], clean[1]) and torch.equal(o[0, :t], clean[0, :t])
    assert bool(o[0, t:].isnan().any(-1).all()) and bool(fs[0].isnan().any()) and not bool(fs[1].isnan().any())


@pytest.mark.parametrize("act,shape", [("bf16", (3, 200, 2, 2, 64, 128)), ("bf16", (3, 300, 2, 1, 128, 64)), ("f32", (3, 45, 2, 2, 32, 32)),
                                       ("bf16", (3, 6, 2, 1, 64, 64))])
def test_nan_of_a_row_stays_out_of_its_neighbours(act, shape):
    """Everything of the middle row is NaN: its neighbours' outputs, states and gradients are as without it
    (the last block of a row is filled up with the next one's tokens)."""
    d = dims(*shape, act)
    x = make(*shape, act, seed=8)
    y = {n: t if n == "log_decay" else t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "do", "init", "dfinal"):
        y[n][1] = float("nan")
    both = [(*forward(z, d), *sm.linear_backward(d, z["q"], z["k"], z["v"], z["log_decay"], z["do"], z["init"], z["dfinal"]).values())
            for z in (x, y)]
    for clean, got in zip(*both):
        assert torch.equal(got[::2], clean[::2]) and not bool(clean.isnan().any())
        assert bool(got[1].isnan().any())


@pytest.mark.parametrize("act,dk,dv", [("bf16", 64, 64), ("f32", 16, 32)])
def test_packed_without_any_token(act, dk, dv):
    """No token rows at all: slots keep their states, or become zeros where nothing is continued."""
    d = dims(3, 0, 2, 2, dk, dv, act)
    q = torch.empty(0, 2 * dk, dtype=d.torch_dtype, device="cuda")
    v = torch.empty(0, 2 * dv, dtype=d.torch_dtype, device="cuda")
    state = torch.randn(4, 2, dv, dk, device="cuda")
    before = state.clone()
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    o = sm.linear_prefill_varlen(d, cu, torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda"),
                                 torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda"), q, q, v, torch.zeros(2, device="cuda"), state)
    before[0] = 0.0
    assert o.shape == (0, 2 * dv) and torch.equal(state, before)


def test_the_binding_checks_types_shapes_and_rows():
    shape = (2, 64, 2, 2, 64, 64)
    d = dims(*shape, "bf16")
    x = make(*shape, "bf16", seed=1)

    def call(**kw):
        y = x | kw
        return sm.linear_prefill(d, y["q"], y["k"], y["v"], y["log_decay"], y["init"])

    call()
    for bad in (dict(q=x["q"].float()), dict(log_decay=x["log_decay"].double()), dict(init=x["init"].bfloat16())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=x["q"][:, :63]), dict(k=x["k"][..., :64]), dict(v=x["v"].transpose(0, 1)), dict(init=x["init"][:1]),
                dict(init=x["init"].transpose(2, 3)), dict(log_decay=x["log_decay"][:1]),
                dict(q=torch.zeros(2, 64, 256, dtype=torch.bfloat16, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    off = torch.zeros(2, 64, 136, dtype=torch.bfloat16, device="cuda")[..., 4:132]      # 8 bytes past a 16-byte boundary
    with pytest.raises(sm.SsdError):
        call(q=off)
    with pytest.raises(sm.SsdError):
        sm.linear_prefill(d, x["q"], x["k"], x["v"], x["log_decay"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sm.linear_prefill(sm.LinearDims(2, 64, 2, 2, 64, 64, act="fp16"), x["q"], x["k"], x["v"], x["log_decay"])
