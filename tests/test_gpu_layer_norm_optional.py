"""Gradients of the layer norm through the C entry with some of its optional outputs left out (needs a B200)."""
import pytest
import torch

from hybrid_mamba_ssm_causal_b200 import ssd_mixer as sm
from tests.test_gpu_layer_norm import check_gradients, make

pytestmark = pytest.mark.gpu

# lane teams, a block a row, four vectors a thread, rows no vector divides, rows too wide for registers
SHAPES = [(33, 8, 128), (300, 1, 2688), (5, 1, 16384), (70, 1, 333), (2, 1, 40000)]


def call(x, dy, w, mean, rstd, groups, dx, dw, db, ws, nbytes):
    rows, C = x.shape
    act = sm.SSD_BF16 if x.dtype == torch.bfloat16 else sm.SSD_F32
    at = [None if t is None else t.data_ptr() for t in (dw, db, ws)]
    st = sm.load_library().ssd_mixer_layer_norm_backward(
        rows, groups, C // groups, act, dy.data_ptr(), C, x.data_ptr(), C, w.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), C, *at, nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == sm.SSD_OK


@pytest.mark.parametrize("rows,groups,width", SHAPES)
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_without_parameter_gradients_no_workspace_is_touched(rows, groups, width, act):
    """dweight and dbias NULL: a small workspace inside a larger buffer, one that starts off any boundary and
    none at all give the same dx, and every byte of the buffer stays."""
    x, dy, w, b = make((rows,), groups, width, act, seed=width)
    _, mean, rstd = sm.layer_norm(x, w, b, groups=groups)
    want = sm.layer_norm_backward(dy, x, w, mean, rstd, groups=groups)
    check_gradients(x, dy, w, mean, rstd, groups, *want)
    need = sm.ssd_mixer_layer_norm_backward_workspace_size(rows, groups, width, act)
    buf = torch.full((need + 4096,), 85, dtype=torch.uint8, device="cuda")     # as large as all partial sums
    for ws, nbytes in ((buf, 16), (buf[4:], 16), (buf, 0), (None, 0)):
        dx = torch.empty_like(x)
        call(x, dy, w, mean, rstd, groups, dx, None, None, ws, nbytes)
        assert torch.equal(dx, want[0]) and bool((buf == 85).all())


@pytest.mark.parametrize("rows,groups,width", SHAPES)
def test_one_parameter_gradient(rows, groups, width):
    x, dy, w, b = make((rows,), groups, width, "f32", seed=width)
    _, mean, rstd = sm.layer_norm(x, w, b, groups=groups)
    want = sm.layer_norm_backward(dy, x, w, mean, rstd, groups=groups)
    need = sm.ssd_mixer_layer_norm_backward_workspace_size(rows, groups, width, "f32")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for only in (1, 2):
        dx, one = torch.empty_like(x), torch.empty_like(w)
        call(x, dy, w, mean, rstd, groups, dx, one if only == 1 else None, one if only == 2 else None, ws, need)
        assert torch.equal(dx, want[0]) and torch.equal(one, want[only])
