"""Packed sequences that are cut into segments, on tensor and on CUDA cores (needs a B200). Bounds:
tests/linear_util.py."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import dims, make
from tests.test_gpu_linear import check_forward

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 4, 2, 64, 128), ("bf16", 2, 2, 128, 128), ("f32", 2, 2, 32, 16)]


def segment_tokens_at_most(d):
    """An upper bound of the call's segments: its workspace holds b + T // segment states of each head, or none where
    T is no longer than a segment."""
    states = sm.ssd_mixer_linear_prefill_varlen_workspace_size(d) // (4 * d.nheads * d.dk * d.dv)
    return min(d.seqlen - 1, d.seqlen // (states - d.batch)) if states > d.batch else d.seqlen


def check_packed(kind, offsets, T, has, seed, poison=None):
    """Sequences between `offsets` (clamped to the T rows) on permuted slots, each against its own fp64 form;
    rows of no sequence keep what they held. `poison`: a sequence of NaN, which is not compared."""
    act, H, G, dk, dv = kind
    b = len(offsets) - 1
    d = dims(b, T, H, G, dk, dv, act)
    x = make(1, T, H, G, dk, dv, act, seed=seed)
    gen = torch.Generator().manual_seed(seed)
    slots = torch.randperm(b + 2, generator=gen)[:b].to(torch.int32)
    state = torch.randn(b + 2, H, dv, dk, generator=gen).cuda()
    before = state.clone()
    at = [min(max(c, 0), T) for c in offsets]
    q, k, v = (x[n][0].clone() for n in ("q", "k", "v"))
    if poison is not None:
        k[at[poison]:at[poison + 1]] = float("nan")
    o = torch.full((T, H * dv), 7.0, dtype=d.torch_dtype, device="cuda")
    sm.linear_prefill_varlen(d, torch.tensor(offsets, dtype=torch.int32, device="cuda"), slots.cuda(),
                             torch.tensor(has, dtype=torch.uint8, device="cuda"), q, k, v, x["log_decay"], state, o=o)
    assert bool((o[:at[0]] == 7.0).all()) and bool((o[at[-1]:] == 7.0).all())
    for i in range(b):
        if i == poison:
            continue
        n, s = at[i + 1] - at[i], int(slots[i])
        if n == 0:
            assert torch.equal(state[s], before[s] if has[i] else torch.zeros_like(before[s])), i
            continue
        y = {m: x[m][:, at[i]:at[i + 1]] for m in ("q", "k", "v")}
        y |= {"log_decay": x["log_decay"], "init": before[s][None] if has[i] else None}
        check_forward(y, dims(1, n, H, G, dk, dv, act), o[at[i]:at[i + 1]][None], state[s][None], d.scale)
    free = sorted(set(range(b + 2)) - set(slots.tolist()))
    assert torch.equal(state[free], before[free])
    return d


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_outside_the_rows_are_clamped(kind):
    """Sequences before the first row and behind the last are empty, however far apart their offsets lie; one
    that is cut into segments stands between them."""
    n = 1500 if kind[0] == "bf16" else 200
    offsets = [-9000, -6000, -3000, -1500, 0, n, n + 4000, n + 9000]
    d = check_packed(kind, offsets, n, [1, 0, 1, 1, 1, 0, 1], seed=3)
    assert segment_tokens_at_most(d) < n


@pytest.mark.parametrize("kind", KINDS)
def test_more_sequences_than_one_block_counts(kind):
    """300 sequences, those that are cut among the first 256, behind them, and the last."""
    long = [1100, 1500, 1030] if kind[0] == "bf16" else [200, 333, 130]
    lens = [2] * 300
    lens[3], lens[270], lens[299] = long
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    d = check_packed(kind, offsets, offsets[-1] + 5, [i % 4 != 2 for i in range(300)], seed=4)
    assert segment_tokens_at_most(d) < sorted(long)[1]       # one of them behind the first 256


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("poison", [None, 1, 2])
@pytest.mark.parametrize("flip", [0, 1])
def test_several_sequences_cut_at_once(kind, poison, flip):
    """Three sequences in segments among short, empty and single-token ones, continuing from their slots and not,
    all compared, or beside one of NaN (a short one, the longest)."""
    lens = [1700, 3, 2600, 0, 1025, 1] if kind[0] == "bf16" else [333, 3, 500, 0, 257, 1]
    offsets = [4]
    for n in lens:
        offsets.append(offsets[-1] + n)
    d = check_packed(kind, offsets, offsets[-1] + 7, [(i // 2 + flip) % 2 for i in range(6)], seed=5 + flip, poison=poison)
    assert segment_tokens_at_most(d) < sorted(lens)[-2]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("has", [0, 1])
def test_one_long_sequence(kind, has):
    """A packed call of one sequence is cut as a single row is."""
    n = 4000 if kind[0] == "bf16" else 700
    d = check_packed(kind, [3, 3 + n], n + 20, [has], seed=6)
    assert segment_tokens_at_most(d) < n
