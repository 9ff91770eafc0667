"""What the linear-attention and layer-norm entry points refuse, before any launch (CPU only: every
call here fails validation, so nothing reaches a GPU)."""
import ctypes
import math

import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import build as build_mod
from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm

FAKE = 1 << 40  # a 256-byte-aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return sm.load_library()


def _dims(**kw):
    base = dict(batch=2, seqlen=64, nheads=4, ngroups=2, dk=64, dv=32, scale=0.5, act="bf16")
    base.update(kw)
    return sm.LinearDims(**base)


def rows(d):
    return [FAKE, d.nheads * d.dk, FAKE, d.ngroups * d.dk, FAKE, d.ngroups * d.dv]


def prefill(lib, d, at=None, put=None, c=None):
    a = rows(d) + [FAKE, None, FAKE, d.nheads * d.dv, FAKE, FAKE, BIG, None]
    if at is not None:
        a[at] = put
    return lib.ssd_mixer_linear_prefill(ctypes.byref(c or d.c()), *a)


def varlen(lib, d, at=None, put=None):
    a = [FAKE, None, None] + rows(d) + [FAKE, FAKE, 8, FAKE, d.nheads * d.dv, FAKE, BIG, None]
    if at is not None:
        a[at] = put
    return lib.ssd_mixer_linear_prefill_varlen(ctypes.byref(d.c()), *a)


def decode(lib, d, at=None, put=None):
    a = rows(d) + [FAKE, FAKE, 8, None, FAKE, d.nheads * d.dv, None]
    if at is not None:
        a[at] = put
    return lib.ssd_mixer_linear_decode_step(ctypes.byref(d.c()), *a)


def backward(lib, d, at=None, put=None):
    H, G = d.nheads, d.ngroups
    a = rows(d) + [FAKE, None, FAKE, H * d.dv, None, FAKE, H * d.dk, FAKE, G * d.dk, FAKE, G * d.dv, None, FAKE, BIG, None]
    if at is not None:
        a[at] = put
    return lib.ssd_mixer_linear_backward(ctypes.byref(d.c()), *a)


BAD_DIMS = [(dict(batch=-1), sm.SSD_ERR_INVALID_ARG), (dict(seqlen=-1), sm.SSD_ERR_INVALID_ARG),
            (dict(nheads=0), sm.SSD_ERR_INVALID_ARG), (dict(ngroups=3), sm.SSD_ERR_INVALID_ARG),
            (dict(ngroups=0), sm.SSD_ERR_INVALID_ARG), (dict(dk=0), sm.SSD_ERR_INVALID_ARG),
            (dict(scale=math.inf), sm.SSD_ERR_INVALID_ARG), (dict(scale=math.nan), sm.SSD_ERR_INVALID_ARG),
            (dict(dk=48), sm.SSD_ERR_UNSUPPORTED), (dict(dv=256), sm.SSD_ERR_UNSUPPORTED), (dict(dv=8), sm.SSD_ERR_UNSUPPORTED),
            (dict(batch=65536), sm.SSD_ERR_UNSUPPORTED), (dict(nheads=1 << 17, ngroups=1), sm.SSD_ERR_UNSUPPORTED),
            (dict(seqlen=1 << 40), sm.SSD_ERR_UNSUPPORTED), (dict(seqlen=(1 << 31) - 1), sm.SSD_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", BAD_DIMS)
def test_bad_dims(lib, bad, status):
    d = _dims(**bad)
    for call in (prefill, varlen, backward):
        if call is varlen and bad == dict(seqlen=(1 << 31) - 1):
            assert call(lib, d) == sm.SSD_ERR_UNSUPPORTED
        assert call(lib, d) == status
    for n in ("prefill", "prefill_varlen", "backward"):
        assert getattr(lib, f"ssd_mixer_linear_{n}_workspace_size")(ctypes.byref(d.c())) == 0
    if "seqlen" not in bad:
        assert decode(lib, _dims(**{"seqlen": 1, **bad})) == status


def test_unknown_type_and_null_dims(lib):
    c = _dims().c()
    c.act = 7
    assert prefill(lib, _dims(), c=c) == sm.SSD_ERR_UNSUPPORTED
    assert lib.ssd_mixer_linear_prefill_workspace_size(None) == 0


def test_decode_takes_one_token(lib):
    assert decode(lib, _dims(seqlen=2)) == sm.SSD_ERR_INVALID_ARG
    assert decode(lib, _dims(seqlen=1), 8, 1) == sm.SSD_ERR_INVALID_ARG       # fewer slots than sequences


@pytest.mark.parametrize("call,required,aligned,strides", [
    (prefill, [0, 2, 4, 6, 8, 10, 11], [0, 2, 4, 7, 8, 10], [1, 3, 5, 9]),
    (varlen, [0, 3, 5, 7, 9, 10, 12, 14], [3, 5, 7, 10, 12], [4, 6, 8, 13]),
    (decode, [0, 2, 4, 6, 7, 10], [0, 2, 4, 7, 10], [1, 3, 5, 11]),
    (backward, [0, 2, 4, 6, 8, 11, 13, 15, 18], [0, 2, 4, 7, 8, 10, 11, 13, 15, 17], [1, 3, 5, 9, 12, 14, 16]),
])
def test_missing_and_misplaced_arguments(lib, call, required, aligned, strides):
    d = _dims(seqlen=1 if call is decode else 64)
    for at in required:
        assert call(lib, d, at, None) == sm.SSD_ERR_INVALID_ARG, at
    for at in aligned:
        assert call(lib, d, at, FAKE + 8) == sm.SSD_ERR_UNSUPPORTED, at
    for at in strides:
        assert call(lib, d, at, 8) == sm.SSD_ERR_UNSUPPORTED, at               # rows that overlap
        assert call(lib, d, at, 4 * 64 + 4) == sm.SSD_ERR_UNSUPPORTED, at      # not a multiple of 16 bytes


@pytest.mark.parametrize("name,call,n", [("prefill", prefill, 12), ("prefill_varlen", varlen, 15), ("backward", backward, 19)])
@pytest.mark.parametrize("shape", [{}, dict(seqlen=5000), dict(batch=1, seqlen=20000, nheads=1, ngroups=1)])
def test_small_or_misaligned_workspace(lib, name, call, n, shape):
    d = _dims(**shape)
    need = getattr(lib, f"ssd_mixer_linear_{name}_workspace_size")(ctypes.byref(d.c()))
    assert need >= 256
    assert call(lib, d, n, need - 1) == sm.SSD_ERR_INVALID_ARG
    assert call(lib, d, n - 1, FAKE + 128) == sm.SSD_ERR_INVALID_ARG


def test_an_empty_batch_needs_no_rows(lib):
    d = _dims(batch=0)
    assert lib.ssd_mixer_linear_prefill(ctypes.byref(d.c()), None, 0, None, 0, None, 0, FAKE, None, None, 0, FAKE, FAKE, BIG,
                                        None) == sm.SSD_OK
    d = _dims(batch=0, seqlen=1)
    assert decode(lib, d, 0, None) == sm.SSD_OK


def norm(lib, rows=4, groups=2, width=64, eps=1e-5, act=sm.SSD_BF16, x=FAKE, x_ld=128, w=FAKE, b=FAKE, y=FAKE, y_ld=128,
         mean=FAKE, rstd=FAKE):
    return lib.ssd_mixer_layer_norm(rows, groups, width, eps, act, x, x_ld, w, b, y, y_ld, mean, rstd, None)


def norm_backward(lib, rows=4, groups=2, width=64, act=sm.SSD_BF16, dy=FAKE, dy_ld=128, x=FAKE, x_ld=128, w=FAKE, mean=FAKE,
                  rstd=FAKE, dx=FAKE, dx_ld=128, dw=FAKE, db=FAKE, ws=FAKE, n=BIG):
    return lib.ssd_mixer_layer_norm_backward(rows, groups, width, act, dy, dy_ld, x, x_ld, w, mean, rstd, dx, dx_ld, dw, db, ws,
                                             n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), sm.SSD_ERR_INVALID_ARG), (dict(groups=0), sm.SSD_ERR_INVALID_ARG), (dict(width=0), sm.SSD_ERR_INVALID_ARG),
    (dict(act=2), sm.SSD_ERR_UNSUPPORTED), (dict(width=1 << 25, x_ld=1 << 27), sm.SSD_ERR_UNSUPPORTED),
    (dict(rows=1 << 31), sm.SSD_ERR_UNSUPPORTED), (dict(x=None), sm.SSD_ERR_INVALID_ARG), (dict(x=FAKE + 1), sm.SSD_ERR_UNSUPPORTED),
    (dict(x_ld=127), sm.SSD_ERR_UNSUPPORTED), (dict(w=FAKE + 2), sm.SSD_ERR_UNSUPPORTED), (dict(mean=FAKE + 2), sm.SSD_ERR_UNSUPPORTED),
])
def test_norm_refusals(lib, bad, status):
    assert norm(lib, **bad) == status
    assert norm_backward(lib, **bad) == status


def test_norm_refusals_of_one_direction(lib):
    assert norm(lib, eps=-1.0) == sm.SSD_ERR_INVALID_ARG
    assert norm(lib, eps=math.nan) == sm.SSD_ERR_INVALID_ARG
    assert norm(lib, y=None) == sm.SSD_ERR_INVALID_ARG
    assert norm(lib, b=FAKE + 1) == sm.SSD_ERR_UNSUPPORTED
    assert norm(lib, y_ld=64) == sm.SSD_ERR_UNSUPPORTED
    for n in ("dy", "mean", "rstd", "dx", "ws"):
        assert norm_backward(lib, **{n: None}) == sm.SSD_ERR_INVALID_ARG, n
    assert norm_backward(lib, dw=FAKE + 2) == sm.SSD_ERR_UNSUPPORTED
    need = lib.ssd_mixer_layer_norm_backward_workspace_size(4, 2, 64, sm.SSD_BF16)
    assert need > 0 and norm_backward(lib, n=need - 1) == sm.SSD_ERR_INVALID_ARG
    assert lib.ssd_mixer_layer_norm_backward_workspace_size(4, 0, 64, sm.SSD_BF16) == 0


def test_the_binding_refuses_cpu_tensors():
    d = _dims(dv=64)
    x = torch.zeros(2, 64, 4 * 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sm.linear_prefill(d, x, x, x, torch.zeros(4))
    with pytest.raises(TypeError):
        sm.linear_decode_step(d, x, x, x, torch.zeros(4), torch.zeros(1))
    with pytest.raises(TypeError):
        sm.linear_backward(d, x, x, x, torch.zeros(4), x)
    with pytest.raises(TypeError):
        sm.layer_norm(x)
    with pytest.raises(TypeError):
        sm.layer_norm_backward(x, x, None, x, x)


# -------------------------------------------------------------- the split of rows into segments
@pytest.mark.parametrize("seg", [128, 384, 1024])
def test_items_of_a_packed_call_are_distinct_and_in_range(seg):
    """Segment t of sequence i is item i + floor(start_i / seg) + t; the state buffer holds b + T / seg
    items, and the kernels find i as the last one with i + floor(start_i / seg) <= item."""
    import random
    rng = random.Random(seg)
    for _ in range(200):
        lens = [rng.choice([0, 1, 2, 127, 128, 129, rng.randrange(3000)]) for _ in range(rng.randrange(1, 12))]
        start, T = [0], sum(lens)
        for n in lens:
            start.append(start[-1] + n)
        seen = {}
        for i, n in enumerate(lens):
            for t in range(max(1, -(-n // seg))):
                item = i + start[i] // seg + t
                assert item not in seen and item < len(lens) + T // seg
                seen[item] = (i, t)
        for item, (i, t) in seen.items():
            lo = max(j for j in range(len(lens)) if j + start[j] // seg <= item)
            assert (lo, item - (lo + start[lo] // seg)) == (i, t)
