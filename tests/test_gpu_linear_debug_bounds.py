"""Linear attention in the bounds-checked build (libssd_mixer_debug.so): rows, slots and segment states of calls of
every kind stay inside their buffers, the status word reads OK and the results are those of the fp64 form (needs a
B200). The calls run in a process of their own, as the binding keeps one library for each."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r'''
import torch
from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.linear_util import dims, make
from tests.test_gpu_linear import check_backward, check_forward
assert sm.load_library()._name.endswith("libssd_mixer_debug.so")

def space(size):
    return torch.full((size,), 255, dtype=torch.uint8, device="cuda")      # the status word holds no code of the library's

def ok(ws):
    torch.cuda.synchronize()
    assert sm.ssd_mixer_workspace_status(ws) == sm.SSD_OK

# tensor cores whole and cut, ragged pieces, shared heads; CUDA cores whole and cut; short rows; no tokens
for shape, act in [((2, 300, 3, 3, 64, 64), "bf16"), ((1, 3001, 2, 1, 128, 128), "bf16"), ((1, 5001, 60, 60, 64, 64), "bf16"),
                   ((2, 700, 2, 2, 128, 64), "bf16"), ((1, 333, 2, 1, 64, 16), "f32"), ((3, 40, 2, 2, 32, 32), "bf16"),
                   ((3, 7, 2, 2, 64, 64), "bf16"), ((2, 0, 2, 2, 64, 64), "bf16")]:
    d, x = dims(*shape, act), make(*shape, act, seed=1)
    ws = space(sm.ssd_mixer_linear_prefill_workspace_size(d))
    o, fs = sm.linear_prefill(d, x["q"], x["k"], x["v"], x["log_decay"], x["init"], workspace=ws)
    ok(ws)
    ws = space(sm.ssd_mixer_linear_backward_workspace_size(d))
    g = sm.linear_backward(d, x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["dfinal"], workspace=ws)
    ok(ws)
    if shape[1] * shape[2] < 10000:
        check_forward(x, d, o, fs, d.scale)
        check_backward(x, d, g)

# packed rows: long, short, empty, on slots, with offsets outside the rows
for act, H, dk, dv, offsets, T in [("bf16", 4, 64, 128, [-3000, 0, 1, 1700, 1703, 4303, 4303, 9000], 4500),
                                   ("f32", 2, 32, 16, [-300, 0, 1, 333, 336, 836, 836, 2000], 900)]:
    b = len(offsets) - 1
    d, x = dims(b, T, H, H, dk, dv, act), make(1, T, H, H, dk, dv, act, seed=2)
    ws = space(sm.ssd_mixer_linear_prefill_varlen_workspace_size(d))
    state = torch.randn(b + 2, H, dv, dk, generator=torch.Generator().manual_seed(2)).cuda()
    before = state.clone()
    slots = torch.tensor([8, 3, 0, -1, 5, 9, 1], dtype=torch.int32, device="cuda")
    o = sm.linear_prefill_varlen(d, torch.tensor(offsets, dtype=torch.int32, device="cuda"), slots, None, x["q"][0], x["k"][0],
                                 x["v"][0], x["log_decay"], state, workspace=ws)
    ok(ws)
    for i, s in enumerate(slots.tolist()):
        at, to = (min(max(offsets[i + j], 0), T) for j in (0, 1))
        if 0 <= s < b + 2 and to > at:
            y = {n: x[n][:, at:to] for n in ("q", "k", "v")} | {"log_decay": x["log_decay"], "init": before[s][None]}
            check_forward(y, dims(1, to - at, H, H, dk, dv, act), o[at:to][None], state[s][None], d.scale)
print("debug-bounds cases ok")
'''


@pytest.mark.gpu
def test_bounds_checked_build_reports_no_violation():
    from hybrid_mamba_ssm_causal_b200 import build
    lib = build.build(debug_bounds=True)
    env = dict(os.environ, SSD_MIXER_LIBRARY=lib)
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "debug-bounds cases ok" in r.stdout


@pytest.mark.parametrize("name", ["ssd_linear.cu", "ssd_linear_tc.cu"])
def test_the_checks_are_compiled_in(name, tmp_path):
    """The flag reaches the scans' sources: preprocessed with it they call the check."""
    from hybrid_mamba_ssm_causal_b200 import build
    texts = []
    for extra in ([], ["-DSSD_DEBUG_BOUNDS"]):
        out = tmp_path / "out.ii"
        subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, *extra, "-E", os.path.join(build.CSRC, name), "-o", str(out)],
                       check=True, capture_output=True, timeout=600)
        texts.append(out.read_text(errors="replace").count("ssd_in_bounds(("))
    assert texts[0] == 0 and texts[1] > 0
