"""Timed cases of linear attention with a decay per head and of layer norm, with their plain forms.

Linear attention (b rows, H heads, key dim dk, value dim dv, k and v shared by groups of H / G
heads, decay lambda_h = exp(log_decay[h]) of head h):
    S_t = lambda S_{t-1} + v_t k_t^T   ([dv, dk], S_{-1} the initial state),   o_t = scale S_t q_t
Layer norm (over each of `groups` contiguous runs of a row's channels):
    y = (x - mean) rstd w + b,   rstd = 1 / sqrt(var + eps)

``run`` computes them with elementary torch operations in fp32 (chunk by chunk, 128 tokens), or,
where ``own`` is true, through the library's entry points. ``exact`` computes the same in fp64 from
the definition written out over all pairs of tokens.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 128
EPS = 1e-5


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a short prompt of a small model: launch latency
        {"name": "prefill_short_bf16", "op": "prefill", "act": "bf16", "b": 1, "L": 96, "H": 8, "G": 8, "dk": 64, "dv": 64,
         "init": False},
        # full precision, uneven lengths and head dims
        {"name": "prefill_f32", "op": "prefill", "act": "f32", "b": 2, "L": 777, "H": 12, "G": 12, "dk": 64, "dv": 32,
         "init": True},
        # one piece of a long-context prompt that continues from a state (the 16384-token pieces of long_bf16)
        {"name": "prefill_long_bf16", "op": "prefill", "act": "bf16", "b": 1, "L": 16384, "H": 64, "G": 64, "dk": 128,
         "dv": 128, "init": True},
        # an engine's mixed batch: prompts of any length and single tokens on their state slots, shared k and v heads
        {"name": "varlen_bf16", "op": "varlen", "act": "bf16", "b": 14, "L": 12289, "H": 32, "G": 8, "dk": 128, "dv": 128,
         "init": True},
        # one sequence decoding: latency
        {"name": "decode_one_bf16", "op": "decode", "act": "bf16", "b": 1, "L": 1, "H": 32, "G": 32, "dk": 128, "dv": 128,
         "init": True},
        # a full decode batch (the state of decode_bf16: 128 heads of 64 by 128)
        {"name": "decode_batch_bf16", "op": "decode", "act": "bf16", "b": 256, "L": 1, "H": 128, "G": 128, "dk": 128,
         "dv": 64, "init": True},
        # training step of a small model, uneven length
        {"name": "backward_small_bf16", "op": "backward", "act": "bf16", "b": 2, "L": 1500, "H": 16, "G": 16, "dk": 64,
         "dv": 64, "init": False},
        # training on long rows with shared k and v heads, states carried between pieces
        {"name": "backward_long_bf16", "op": "backward", "act": "bf16", "b": 1, "L": 8192, "H": 32, "G": 8, "dk": 128,
         "dv": 128, "init": True},
        # a decode batch's pre-norm
        {"name": "norm_decode_bf16", "op": "norm", "act": "bf16", "rows": 256, "groups": 1, "width": 2688},
        # the norm of a long prefill's attention output, per head
        {"name": "norm_heads_bf16", "op": "norm", "act": "bf16", "rows": 32768, "groups": 64, "width": 128},
        # training in full precision, mid_bf16's model width
        {"name": "norm_backward_f32", "op": "norm_backward", "act": "f32", "rows": 2048, "groups": 1, "width": 2688},
        # training batch of a wide model
        {"name": "norm_backward_bf16", "op": "norm_backward", "act": "bf16", "rows": 16384, "groups": 1, "width": 8192},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "varlen", "decode", "backward", "norm", "norm_backward"])
    if op in ("norm", "norm_backward"):
        act = rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.3:      # per-head norms
            groups, width = rng.choice([4, 8, 12, 32, 64]), rng.choice([64, 128, 256])
        else:
            groups, width = 1, rng.choice([8, 4]) * _log(rng, 16, 1100)
        most = min(32768, (1 << 26) // (groups * width))
        return {"op": op, "act": act, "rows": _log(rng, 1, most), "groups": groups, "width": width}
    act = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "varlen":
        act = "bf16" if rng.random() < 0.8 else "f32"
    dims = [64, 128] if act == "bf16" and rng.random() < 0.8 else [16, 32, 64, 128]
    dk, dv = rng.choice(dims), rng.choice(dims)
    G = _log(rng, 1, 16)
    H = G * rng.choice([1, 1, 1, 2, 4])
    if op == "decode":
        return {"op": op, "act": act, "b": _log(rng, 1, 256), "L": 1, "H": H, "G": G, "dk": dk, "dv": dv, "init": True}
    b = _log(rng, 1, 8) if op != "varlen" else _log(rng, 1, 24)
    most = 16384 * 64 if act == "bf16" else 32768      # token-heads of a call
    L = _log(rng, 1, max(1, min(16384, most // (2 * H * (b if op != "varlen" else 1)))))
    return {"op": op, "act": act, "b": b, "L": L, "H": H, "G": G, "dk": dk, "dv": dv, "init": rng.random() < 0.5}


def work(case):
    es = 2 if case["act"] == "bf16" else 4
    if case["op"] in ("norm", "norm_backward"):
        n, g = case["rows"] * case["groups"] * case["width"], case["rows"] * case["groups"]
        c = case["groups"] * case["width"]
        if case["op"] == "norm":
            return {"bytes": 2 * n * es + 8 * c + 8 * g, "flops": 8 * n}
        return {"bytes": 3 * n * es + 12 * c + 8 * g, "flops": 14 * n}
    H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
    T = case["L"] if case["op"] == "varlen" else case["b"] * case["L"]
    state = 4 * case["b"] * H * dk * dv
    q, kv = T * H * dk * es, T * G * (dk + dv) * es
    o = T * H * dv * es
    if case["op"] == "backward":
        return {"bytes": 2 * q + o + 2 * kv + (3 if case["init"] else 1) * state, "flops": 10 * T * H * dk * dv}
    reads = 1 if case["init"] else 0
    return {"bytes": q + kv + o + (1 + reads) * state, "flops": 4 * T * H * dk * dv}


# ------------------------------------------------------------------------------- inputs
def _act(case):
    return torch.bfloat16 if case["act"] == "bf16" else torch.float32


def _lengths(case):
    """Sequence lengths of a packed batch, set by the case alone: single tokens, an empty one, uneven prompts."""
    b, T = case["b"], case["L"]
    r = np.random.RandomState(1000 * b + T % 1000)
    cut = np.sort(r.randint(0, T + 1, b - 1)) if b > 1 else np.zeros(0, np.int64)
    if b > 4 and T > 8:
        cut[0], cut[1] = 1, 2                 # two sequences of one token
        cut[2] = max(2, cut[2])
        cut[3] = cut[2]                       # an empty one
        cut = np.sort(cut)
    return np.diff(np.concatenate([[0], cut, [T]])).astype(np.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    a = _act(case)
    s = {"case": case}
    if case["op"] in ("norm", "norm_backward"):
        rows, groups, width = case["rows"], case["groups"], case["width"]
        c = groups * width
        # hidden states: an offset and a scale of each channel, a scale of each row
        x = normal(rows, c)
        x.mul_(torch.exp(0.5 * normal(1, c))).add_(0.5 * normal(1, c)).mul_(torch.exp(0.3 * normal(rows, 1)))
        s["x"] = x.to(a)
        s["w"], s["bias"] = 1 + 0.1 * normal(c), 0.1 * normal(c)
        if case["op"] == "norm_backward":
            s["dy"] = normal(rows, c, dtype=a)
            xg = s["x"].view(rows, groups, width).double()
            s["mean"] = xg.mean(-1).float()
            s["rstd"] = (xg.var(-1, unbiased=False) + EPS).rsqrt().float()
        return s
    b, H, G, dk, dv = case["b"], case["H"], case["G"], case["dk"], case["dv"]
    lead = (case["L"],) if case["op"] == "varlen" else (b,) if case["op"] == "decode" else (b, case["L"])
    s["q"], s["k"], s["v"] = normal(*lead, H * dk, dtype=a), normal(*lead, G * dk, dtype=a), normal(*lead, G * dv, dtype=a)
    # decays from exp(-1) to exp(-1/256), as spread over the heads, each moved a little by the seed
    slope = 2.0 ** (-8.0 * torch.arange(H, device="cuda") / max(1, H - 1))
    s["log_decay"] = (-slope * torch.exp(0.1 * normal(H))).contiguous()
    s["scale"] = dk ** -0.5
    if case["op"] in ("varlen", "decode"):
        slots = b + 3
        s["state"] = normal(slots, H, dv, dk)
        s["slot_idx"] = torch.randperm(slots, generator=gen, device="cuda")[:b].to(torch.int32)
        if case["op"] == "varlen":
            lens = _lengths(case)
            s["longest"] = int(lens.max())
            s["cu_seqlens"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
            s["has_init"] = (torch.arange(b, device="cuda") % 3 != 1).to(torch.uint8) if case["init"] else torch.zeros(
                b, dtype=torch.uint8, device="cuda")
    else:
        s["init"] = normal(b, H, dv, dk) if case["init"] else None
        if case["op"] == "backward":
            s["do"] = normal(b, case["L"], H * dv, dtype=a)
            s["dfinal"] = normal(b, H, dv, dk) if case["init"] else None
    return s


# ------------------------------------------------------------------------------- plain forms
def _decay_power(log_decay, n):
    """lambda^n for whole n >= 0 of any shape, heads first; the exponent's product in fp64."""
    return torch.exp(log_decay.double().view(-1, *([1] * n.dim())) * n.double()).float()


def _heads(t, n, d, H):
    """[..., n * d] as fp32 [b, H, L, d], shared heads repeated."""
    t = t.float().unflatten(-1, (n, d)).transpose(-3, -2)
    return t.repeat_interleave(H // n, dim=-3) if H != n else t


def _plain_scan(q, k, v, log_decay, init, init_power, end_power):
    """Decayed causal products of [b, H, L, .] fp32: o_t = sum_{j<=t} lambda^{t-j} (q_t k_j) v_j +
    lambda^{init_power[t]} init q_t, and the state sum_j lambda^{L-1-j} v_j k_j^T + lambda^{end_power} init."""
    b, H, L, dk = q.shape
    dv = v.shape[-1]
    nc = max(1, -(-L // CHUNK))
    pad = nc * CHUNK - L                     # padding in front, so that the last chunk ends with the row
    qc, kc, vc = (torch.nn.functional.pad(t, (0, 0, pad, 0)).view(b, H, nc, CHUNK, -1) for t in (q, k, v))
    i = torch.arange(CHUNK, device=q.device)
    gap = i[:, None] - i[None, :]
    inside = _decay_power(log_decay, gap.clamp(min=0)) * (gap >= 0)                      # [H, C, C]
    o = ((qc @ kc.transpose(-1, -2)) * inside[None, :, None]) @ vc
    added = (vc * _decay_power(log_decay, CHUNK - 1 - i)[None, :, None, :, None]).transpose(-1, -2) @ kc   # [b,H,nc,dv,dk]
    c = torch.arange(nc, device=q.device)
    cgap = c[:, None] - 1 - c[None, :]
    between = _decay_power(log_decay, CHUNK * cgap.clamp(min=0)) * (cgap >= 0)           # [H, nc, nc]
    entering = (between @ added.flatten(-2)).view(b, H, nc, dv, dk)
    o = o + _decay_power(log_decay, i + 1)[None, :, None, :, None] * (qc @ entering.transpose(-1, -2))
    last = _decay_power(log_decay, torch.tensor(CHUNK, device=q.device)).view(1, H, 1, 1)
    final = last * entering[:, :, -1] + added[:, :, -1]
    o = o.view(b, H, nc * CHUNK, dv)[:, :, pad:]
    if init is not None:
        o = o + init_power[..., None] * (q @ init.transpose(-1, -2))
        final = final + end_power * init
    return o, final


def _rows(o, dtype):
    """[b, H, L, d] to [b, L, H * d] in the activations' type."""
    return o.transpose(1, 2).flatten(2).to(dtype)


def _plain_prefill(s):
    case = s["case"]
    H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
    g, L = s["log_decay"], case["L"]
    t = torch.arange(L, device="cuda")
    o, final = _plain_scan(_heads(s["q"], H, dk, H), _heads(s["k"], G, dk, H), _heads(s["v"], G, dv, H), g, s["init"],
                           _decay_power(g, t + 1), _decay_power(g, torch.tensor(L, device="cuda")).view(H, 1, 1))
    return [_rows(s["scale"] * o, s["q"].dtype), final]


def _plain_varlen(s):
    case = s["case"]
    H, G, dk, dv, b = case["H"], case["G"], case["dk"], case["dv"], case["b"]
    g, Lm = s["log_decay"], s["longest"]
    cu = s["cu_seqlens"].long()
    lens = cu[1:] - cu[:-1]
    t = torch.arange(Lm, device="cuda")[None] - (Lm - lens)[:, None]            # [b, Lm]; rows end together
    row = (cu[:-1, None] + t).clamp(min=0, max=max(0, case["L"] - 1))
    used = (t >= 0)
    q, k, v = ((s[n][row] * used[..., None]) for n in ("q", "k", "v"))
    slot = s["slot_idx"].long()
    init = s["state"][slot] * s["has_init"].view(b, 1, 1, 1)
    power = _decay_power(g, (t + 1).clamp(min=0)).transpose(0, 1)               # [b, H, Lm]
    end = _decay_power(g, lens).transpose(0, 1)[..., None, None]
    o, final = _plain_scan(_heads(q, H, dk, H), _heads(k, G, dk, H), _heads(v, G, dv, H), g, init, power, end)
    out = torch.empty(case["L"], H * dv, dtype=s["q"].dtype, device="cuda")
    out[row[used]] = _rows(s["scale"] * o, out.dtype)[used]
    s["state"][slot] = final
    return [out, s["state"]]


def _plain_decode(s):
    case = s["case"]
    H, G, dk, dv, b = case["H"], case["G"], case["dk"], case["dv"], case["b"]
    slot = s["slot_idx"].long()
    q, k, v = (_heads(s[n].view(b, 1, -1), m, d, H)[:, :, 0] for n, m, d in (("q", H, dk), ("k", G, dk), ("v", G, dv)))
    S = torch.exp(s["log_decay"]).view(1, H, 1, 1) * s["state"][slot] + v[..., :, None] * k[..., None, :]
    s["state"][slot] = S
    o = s["scale"] * (S * q[..., None, :]).sum(-1)
    return [o.flatten(1).to(s["q"].dtype), s["state"]]


def _plain_backward(s):
    case = s["case"]
    H, G, dk, dv, L, b = case["H"], case["G"], case["dk"], case["dv"], case["L"], case["b"]
    g, scale, a = s["log_decay"], s["scale"], s["q"].dtype
    q, k, v = _heads(s["q"], H, dk, H), _heads(s["k"], G, dk, H), _heads(s["v"], G, dv, H)
    do = _heads(s["do"], H, dv, H)
    t = torch.arange(L, device="cuda")
    none = _decay_power(g, torch.tensor(L, device="cuda")).view(H, 1, 1)
    init_t = None if s["init"] is None else s["init"].transpose(-1, -2)
    dq, _ = _plain_scan(do, v, k, g, init_t, _decay_power(g, t + 1), none)
    # dk and dv: the same sums over the tokens that follow
    qr, kr, vr, dor = (x.flip(2) for x in (scale * q, k, v, do))
    back = None if s["dfinal"] is None else s["dfinal"].transpose(-1, -2)
    end = _decay_power(g, torch.tensor(max(L - 1, 0), device="cuda")).view(H, 1, 1)
    dk_, _ = _plain_scan(vr, dor, qr, g, back, _decay_power(g, t), end)
    dv_, back_state = _plain_scan(kr, qr, dor, g, s["dfinal"], _decay_power(g, t), end)
    decay = torch.exp(g).view(1, H, 1, 1)
    shared = [x.flip(2).view(b, G, H // G, L, -1).sum(2) for x in (dk_, dv_)]
    return [_rows(scale * dq, a), _rows(shared[0], a), _rows(shared[1], a), decay * back_state]


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float().view(c["rows"], c["groups"], c["width"])
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = torch.rsqrt((d * d).mean(-1) + EPS)
    y = (d * rstd[..., None]).flatten(1) * s["w"] + s["bias"]
    return [y.to(s["x"].dtype), mean, rstd]


def _plain_norm_backward(s):
    c = s["case"]
    shape = (c["rows"], c["groups"], c["width"])
    dy = s["dy"].float()
    xh = (s["x"].float().view(shape) - s["mean"][..., None]) * s["rstd"][..., None]
    dh = (dy * s["w"]).view(shape)
    dx = s["rstd"][..., None] * (dh - dh.mean(-1, keepdim=True) - xh * (dh * xh).mean(-1, keepdim=True))
    return [dx.flatten(1).to(s["x"].dtype), (dy * xh.flatten(1)).sum(0), dy.sum(0)]


# ------------------------------------------------------------------------------- the library's calls
def _dims(s):
    from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
    c = s["case"]
    return sm, sm.LinearDims(batch=c["b"], seqlen=c["L"], nheads=c["H"], ngroups=c["G"], dk=c["dk"], dv=c["dv"],
                             scale=s["scale"], act=c["act"])


def _own_run(s):
    op = s["case"]["op"]
    if op in ("norm", "norm_backward"):
        from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
        if op == "norm":
            return list(sm.layer_norm(s["x"], s["w"], s["bias"], groups=s["case"]["groups"], eps=EPS))
        return list(sm.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], groups=s["case"]["groups"]))
    sm, d = _dims(s)
    if op == "prefill":
        return list(sm.linear_prefill(d, s["q"], s["k"], s["v"], s["log_decay"], s["init"]))
    if op == "varlen":
        o = sm.linear_prefill_varlen(d, s["cu_seqlens"], s["slot_idx"], s["has_init"], s["q"], s["k"], s["v"],
                                     s["log_decay"], s["state"])
        return [o, s["state"]]
    if op == "decode":
        o = sm.linear_decode_step(d, s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["slot_idx"])
        return [o, s["state"]]
    r = sm.linear_backward(d, s["q"], s["k"], s["v"], s["log_decay"], s["do"], s["init"], s["dfinal"])
    return [r["q"], r["k"], r["v"], r["init_state"]]


_PLAIN = {"prefill": _plain_prefill, "varlen": _plain_varlen, "decode": _plain_decode, "backward": _plain_backward,
          "norm": _plain_norm, "norm_backward": _plain_norm_backward}


def run(s):
    if own:
        return _own_run(s)
    return _PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------------------- fp64
def _exact_attention(q, k, v, g, init, scale):
    """One sequence of one head in fp64, over all pairs of tokens, a band of query rows at a time."""
    L = q.shape[0]
    j = torch.arange(L, device=q.device, dtype=torch.float64)
    out = []
    for t0 in range(0, L, 4096):
        t1 = min(L, t0 + 4096)
        w = torch.exp(g * (j[t0:t1, None] - j[None, :t1]).clamp(min=0)).tril(t0)
        o = scale * ((q[t0:t1] @ k[:t1].T) * w) @ v[:t1]
        if init is not None:
            o += scale * torch.exp(g * (j[t0:t1] + 1))[:, None] * (q[t0:t1] @ init.T)
        out.append(o)
    final = (v * torch.exp(g * (L - 1 - j))[:, None]).T @ k
    if init is not None:
        final = final + math.exp(g * L) * init
    return (torch.cat(out) if out else v[:0]), final


def _exact_gradients(q, k, v, do, g, init, dfinal, scale):
    L = q.shape[0]
    j = torch.arange(L, device=q.device, dtype=torch.float64)
    dq, dk, dv = [], torch.zeros_like(k), torch.zeros_like(v)
    for t0 in range(0, L, 4096):
        t1 = min(L, t0 + 4096)
        w = scale * torch.exp(g * (j[t0:t1, None] - j[None, :t1]).clamp(min=0)).tril(t0)
        p, dp = (q[t0:t1] @ k[:t1].T) * w, (do[t0:t1] @ v[:t1].T) * w
        dq.append(dp @ k[:t1])
        dk[:t1] += dp.T @ q[t0:t1]
        dv[:t1] += p.T @ do[t0:t1]
    dq = torch.cat(dq)
    dinit = scale * (do * torch.exp(g * (j + 1))[:, None]).T @ q
    if init is not None:
        dq += scale * torch.exp(g * (j + 1))[:, None] * (do @ init)
    if dfinal is not None:
        left = torch.exp(g * (L - 1 - j))[:, None]
        dk += left * (v @ dfinal)
        dv += left * (k @ dfinal.T)
        dinit = dinit + math.exp(g * L) * dfinal
    return dq, dk, dv, dinit


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        outs = []
        rows, groups, width = case["rows"], case["groups"], case["width"]
        x = s["x"].double().view(rows, groups, width)
        if op == "norm":
            var, mean = torch.var_mean(x, dim=-1, unbiased=False)
            rstd = 1.0 / torch.sqrt(var + EPS)
            y = (x - mean[..., None]) * rstd[..., None]
            return [y.reshape(rows, -1) * s["w"].double() + s["bias"].double(), mean, rstd]
        dy, w = s["dy"].double().view(rows, groups, width), s["w"].double().view(1, groups, width)
        mean, rstd = s["mean"].double()[..., None], s["rstd"].double()[..., None]
        x.sub_(mean).mul_(rstd)                                      # normalised
        dw, db = torch.einsum("rgw,rgw->gw", dy, x), dy.sum(0)
        m2 = torch.einsum("rgw,rgw,gw->rg", dy, x, w[0])[..., None] / width
        dy.mul_(w)
        m1 = dy.sum(-1, keepdim=True) / width
        outs = [(dy.sub_(m1).sub_(x.mul_(m2)).mul_(rstd)).reshape(rows, -1), dw.reshape(-1), db.reshape(-1)]
        return outs
    H, G, dk, dv, b = case["H"], case["G"], case["dk"], case["dv"], case["b"]
    r, scale = H // G, s["scale"]
    g = s["log_decay"].double().tolist()
    if op == "decode":
        out = torch.empty(b, H, dv, dtype=torch.float64, device="cuda")
        state = s["state"].double()
        q, k, v = (s[n].double().view(b, m, d) for n, m, d in (("q", H, dk), ("k", G, dk), ("v", G, dv)))
        at = s["slot_idx"].long()
        for h in range(H):
            one = torch.exp(s["log_decay"][h].double()) * state[at, h] + torch.einsum("bd,be->bde", v[:, h // r], k[:, h // r])
            state[at, h] = one
            out[:, h] = scale * torch.einsum("bde,be->bd", one, q[:, h])
        return [out.view(b, H * dv), state]
    if op == "varlen":
        cu, slots, has = s["cu_seqlens"].tolist(), s["slot_idx"].tolist(), s["has_init"].tolist()
        out = torch.empty(case["L"], H, dv, dtype=torch.float64, device="cuda")
        state = s["state"].double()
        q, k, v = (s[n].double().view(-1, m, d) for n, m, d in (("q", H, dk), ("k", G, dk), ("v", G, dv)))
        for i in range(b):
            at = slice(cu[i], cu[i + 1])
            for h in range(H):
                init = state[slots[i], h].clone() if has[i] else None
                out[at, h], state[slots[i], h] = _exact_attention(q[at, h], k[at, h // r], v[at, h // r], g[h], init, scale)
        return [out.view(case["L"], H * dv), state]
    L = case["L"]
    q, k, v = (s[n].double().view(b, L, m, d) for n, m, d in (("q", H, dk), ("k", G, dk), ("v", G, dv)))
    if op == "prefill":
        out = torch.empty(b, L, H, dv, dtype=torch.float64, device="cuda")
        state = torch.empty(b, H, dv, dk, dtype=torch.float64, device="cuda")
        for i in range(b):
            for h in range(H):
                init = s["init"][i, h].double() if s["init"] is not None else None
                out[i, :, h], state[i, h] = _exact_attention(q[i, :, h], k[i, :, h // r], v[i, :, h // r], g[h], init, scale)
        return [out.view(b, L, H * dv), state]
    do = s["do"].double().view(b, L, H, dv)
    dq, dk_, dv_ = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dinit = torch.empty(b, H, dv, dk, dtype=torch.float64, device="cuda")
    for i in range(b):
        for h in range(H):
            init, dfinal = (None if s[n] is None else s[n][i, h].double() for n in ("init", "dfinal"))
            one = _exact_gradients(q[i, :, h], k[i, :, h // r], v[i, :, h // r], do[i, :, h], g[h], init, dfinal, scale)
            dq[i, :, h], dinit[i, h] = one[0], one[3]
            dk_[i, :, h // r] += one[1]
            dv_[i, :, h // r] += one[2]
    return [dq.view(b, L, -1), dk_.view(b, L, -1), dv_.view(b, L, -1), dinit]
