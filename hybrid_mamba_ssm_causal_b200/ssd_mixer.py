"""Thin Python binding of the C ABI in include/ssd_mixer.h (argument marshalling only).

Every step of the mixer runs in libssd_mixer.so; this module only turns torch tensors
into device pointers, leading dimensions and the current CUDA stream. There is no
fallback: if the library is missing or the tensors are not on a CUDA device, the call
raises.

The entry points keep the C names:
  ssd_mixer_prefill_workspace_size(dims) -> int
  ssd_mixer_prefill(dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                    init_ssm_state, init_conv_state, y, final_ssm_state, final_conv_state,
                    workspace, stream=None)
  ssd_mixer_decode_step(dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                        ssm_state, conv_state, slot_idx, y, stream=None)
  ssd_mixer_backward(dims, <prefill inputs>, dy, dfinal_ssm_state, dfinal_conv_state,
                     <gradients>, workspace, stream=None)
plus :func:`prefill` / :func:`decode_step` / :func:`backward`, which allocate the outputs
and workspace with torch and call the entry points above.

Linear attention with a decay per head (:class:`LinearDims`, :func:`linear_prefill`,
:func:`linear_prefill_varlen`, :func:`linear_decode_step`, :func:`linear_backward`) and the
grouped layer norm (:func:`layer_norm`, :func:`layer_norm_backward`) check every tensor's type,
shape and device, run on the device of their inputs whichever is current, and allocate what is
not given. Unless ``stream`` (a torch stream or a handle) is given, they run on that device's
current stream. A call's status word (:func:`ssd_mixer_workspace_status`) can be read where
``workspace`` was given.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# the library the binding opens: libssd_mixer.so, or another build of it (the bounds-checked
# libssd_mixer_debug.so) named by SSD_MIXER_LIBRARY
LIB_PATH = os.environ.get("SSD_MIXER_LIBRARY") or os.path.join(HERE, "libssd_mixer.so")

SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_CUDA, SSD_ERR_TIMEOUT, SSD_ERR_TOO_LARGE, SSD_ERR_DEVICE = range(7)
SSD_MIXER_STATIC_WORKSPACE_BYTES = 64 * 1024 * 1024
SSD_F32, SSD_BF16 = 0, 1
SYMBOLS = ("ssd_mixer_prefill_workspace_size", "ssd_mixer_prefill", "ssd_mixer_decode_step",
           "ssd_mixer_workspace_status", "ssd_status_string", "ssd_mixer_version",
           "ssd_mixer_launch_count", "ssd_mixer_profile_enable", "ssd_mixer_profile_read",
           "ssd_mixer_prefill_static", "ssd_mixer_prefill_varlen_workspace_size", "ssd_mixer_prefill_varlen",
           "ssd_mixer_prefill_state_workspace_size", "ssd_mixer_prefill_state", "ssd_mixer_state_pass",
           "ssd_mixer_backward_workspace_size", "ssd_mixer_backward", "ssd_mixer_selftest_wait",
           "ssd_mixer_prefill_static_status", "ssd_mixer_prefill_path", "ssd_mixer_prefill_plan",
           "ssd_mixer_prefill_stage_offsets",
           "ssd_mixer_projection", "ssd_mixer_layer_workspace_size", "ssd_mixer_layer_prefill",
           "ssd_mixer_linear_prefill_workspace_size", "ssd_mixer_linear_prefill",
           "ssd_mixer_linear_prefill_varlen_workspace_size", "ssd_mixer_linear_prefill_varlen",
           "ssd_mixer_linear_decode_step", "ssd_mixer_linear_backward_workspace_size", "ssd_mixer_linear_backward",
           "ssd_mixer_layer_norm", "ssd_mixer_layer_norm_backward_workspace_size", "ssd_mixer_layer_norm_backward")
SSD_PATH_NONE, SSD_PATH_CUDA_CORES, SSD_PATH_TENSOR_CORES = range(3)


class SsdError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class _CDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("dstate", ctypes.c_int32),
                ("dconv", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("eps", ctypes.c_float), ("act", ctypes.c_int32)]


@dataclass(frozen=True)
class Dims:
    batch: int
    seqlen: int
    nheads: int
    headdim: int
    ngroups: int
    dstate: int
    chunk: int = 128
    dconv: int = 4
    eps: float = 1e-5
    act: str = "bf16"

    @property
    def d_inner(self) -> int:
        return self.nheads * self.headdim

    @property
    def xbc_channels(self) -> int:
        return self.d_inner + 2 * self.ngroups * self.dstate

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.act == "bf16" else torch.float32

    def c(self) -> _CDims:
        return _CDims(self.batch, self.seqlen, self.nheads, self.headdim, self.ngroups,
                      self.dstate, self.dconv, self.chunk, self.eps,
                      SSD_BF16 if self.act == "bf16" else SSD_F32)


class _CLinearDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("scale", ctypes.c_float), ("act", ctypes.c_int32)]


@dataclass(frozen=True)
class LinearDims:
    """Sizes of a linear-attention call: batch rows (or packed sequences) of seqlen tokens (packed
    call: token rows in all; decode: 1), nheads heads, ngroups heads of k and v."""
    batch: int
    seqlen: int
    nheads: int
    ngroups: int
    dk: int
    dv: int
    scale: float = 1.0
    act: str = "bf16"

    @property
    def torch_dtype(self):
        return _ACT_DTYPES[self.act]

    def c(self) -> _CLinearDims:
        return _CLinearDims(self.batch, self.seqlen, self.nheads, self.ngroups, self.dk, self.dv, self.scale,
                            SSD_BF16 if self.act == "bf16" else SSD_F32)


_ACT_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

_lib = None


def load_library(path: str = LIB_PATH):
    """Open libssd_mixer.so (raises if it is absent: build it with
    ``python -m hybrid_mamba_ssm_causal_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing "
                           "(run python -m hybrid_mamba_ssm_causal_b200.build)")
    lib = ctypes.CDLL(path)
    V, I64, P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p
    FP = ctypes.c_void_p
    lib.ssd_mixer_prefill_workspace_size.argtypes = [ctypes.POINTER(_CDims)]
    lib.ssd_mixer_prefill_workspace_size.restype = ctypes.c_size_t
    lib.ssd_mixer_prefill.argtypes = ([ctypes.POINTER(_CDims)] + [P, I64] * 5 + [FP] * 6 +
                                      [FP, P, P, I64, FP, P, P, ctypes.c_size_t, V])
    lib.ssd_mixer_prefill.restype = ctypes.c_int
    lib.ssd_mixer_decode_step.argtypes = ([ctypes.POINTER(_CDims)] + [P, I64] * 5 + [FP] * 6 +
                                          [FP, P, P, P, I64, V])
    lib.ssd_mixer_decode_step.restype = ctypes.c_int
    lib.ssd_mixer_prefill_static.argtypes = ([ctypes.POINTER(_CDims)] + [P, I64] * 5 + [FP] * 6 +
                                             [FP, P, P, I64, FP, P, V])
    lib.ssd_mixer_prefill_static.restype = ctypes.c_int
    lib.ssd_mixer_projection.argtypes = [I64, I64, I64, P, I64, P, I64, P, I64, P, V]
    lib.ssd_mixer_projection.restype = ctypes.c_int
    lib.ssd_mixer_layer_workspace_size.argtypes = [ctypes.POINTER(_CDims), I64]
    lib.ssd_mixer_layer_workspace_size.restype = ctypes.c_size_t
    lib.ssd_mixer_layer_prefill.argtypes = ([ctypes.POINTER(_CDims), I64, P, I64, P, P] + [FP] * 6 +
                                            [FP, P, P, I64, FP, P, ctypes.c_int, P, ctypes.c_size_t, V])
    lib.ssd_mixer_layer_prefill.restype = ctypes.c_int
    lib.ssd_mixer_prefill_path.argtypes = [ctypes.POINTER(_CDims)]
    lib.ssd_mixer_prefill_path.restype = ctypes.c_int
    IP = ctypes.POINTER(ctypes.c_int)
    lib.ssd_mixer_prefill_plan.argtypes = [ctypes.POINTER(_CDims), ctypes.c_int, IP, IP, IP, IP]
    lib.ssd_mixer_prefill_plan.restype = ctypes.c_int
    SZP = ctypes.POINTER(ctypes.c_size_t)
    lib.ssd_mixer_prefill_stage_offsets.argtypes = [ctypes.POINTER(_CDims), SZP, SZP, SZP]
    lib.ssd_mixer_prefill_stage_offsets.restype = ctypes.c_int
    lib.ssd_mixer_prefill_static_status.argtypes = [V]
    lib.ssd_mixer_prefill_static_status.restype = ctypes.c_int
    lib.ssd_mixer_prefill_varlen_workspace_size.argtypes = [ctypes.POINTER(_CDims)]
    lib.ssd_mixer_prefill_varlen_workspace_size.restype = ctypes.c_size_t
    lib.ssd_mixer_prefill_varlen.argtypes = ([ctypes.POINTER(_CDims), P, P, P] + [P, I64] * 5 + [FP] * 6 +
                                             [FP, P, P, I64, P, ctypes.c_size_t, V])
    lib.ssd_mixer_prefill_varlen.restype = ctypes.c_int
    lib.ssd_mixer_prefill_state_workspace_size.argtypes = [ctypes.POINTER(_CDims)]
    lib.ssd_mixer_prefill_state_workspace_size.restype = ctypes.c_size_t
    lib.ssd_mixer_prefill_state.argtypes = ([ctypes.POINTER(_CDims)] + [P, I64] * 4 + [FP] * 4 +
                                            [FP, P, FP, P, FP, P, ctypes.c_size_t, V])
    lib.ssd_mixer_prefill_state.restype = ctypes.c_int
    lib.ssd_mixer_state_pass.argtypes = [I64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                         FP, FP, FP, FP, V]
    lib.ssd_mixer_state_pass.restype = ctypes.c_int
    lib.ssd_mixer_backward_workspace_size.argtypes = [ctypes.POINTER(_CDims)]
    lib.ssd_mixer_backward_workspace_size.restype = ctypes.c_size_t
    lib.ssd_mixer_backward.argtypes = ([ctypes.POINTER(_CDims)] + [P, I64] * 5 + [FP] * 6 + [FP, P] +
                                       [P, I64, FP, FP] + [P, I64] * 5 + [FP] * 8 + [P, ctypes.c_size_t, V])
    lib.ssd_mixer_backward.restype = ctypes.c_int
    LD, I32, SZ = ctypes.POINTER(_CLinearDims), ctypes.c_int32, ctypes.c_size_t
    for n in ("prefill", "prefill_varlen", "backward"):
        f = getattr(lib, f"ssd_mixer_linear_{n}_workspace_size")
        f.argtypes, f.restype = [LD], SZ
    lib.ssd_mixer_linear_prefill.argtypes = [LD] + [P, I64] * 3 + [FP, FP, P, I64, FP, P, SZ, V]
    lib.ssd_mixer_linear_prefill.restype = ctypes.c_int
    lib.ssd_mixer_linear_prefill_varlen.argtypes = [LD, P, P, P] + [P, I64] * 3 + [FP, FP, I64, P, I64, P, SZ, V]
    lib.ssd_mixer_linear_prefill_varlen.restype = ctypes.c_int
    lib.ssd_mixer_linear_decode_step.argtypes = [LD] + [P, I64] * 3 + [FP, FP, I64, P, P, I64, V]
    lib.ssd_mixer_linear_decode_step.restype = ctypes.c_int
    lib.ssd_mixer_linear_backward.argtypes = ([LD] + [P, I64] * 3 + [FP, FP, P, I64, FP] + [P, I64] * 3 +
                                              [FP, P, SZ, V])
    lib.ssd_mixer_linear_backward.restype = ctypes.c_int
    lib.ssd_mixer_layer_norm.argtypes = [I64, I32, I32, ctypes.c_float, I32, P, I64, FP, FP, P, I64, FP, FP, V]
    lib.ssd_mixer_layer_norm.restype = ctypes.c_int
    lib.ssd_mixer_layer_norm_backward_workspace_size.argtypes = [I64, I32, I32, I32]
    lib.ssd_mixer_layer_norm_backward_workspace_size.restype = SZ
    lib.ssd_mixer_layer_norm_backward.argtypes = [I64, I32, I32, I32, P, I64, P, I64, FP, FP, FP, P, I64, FP, FP, P, SZ, V]
    lib.ssd_mixer_layer_norm_backward.restype = ctypes.c_int
    lib.ssd_mixer_selftest_wait.argtypes = [P, ctypes.c_longlong, ctypes.c_int, V]
    lib.ssd_mixer_selftest_wait.restype = ctypes.c_int
    lib.ssd_mixer_workspace_status.argtypes = [P, V]
    lib.ssd_mixer_workspace_status.restype = ctypes.c_int
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_mixer_version.argtypes = []
    lib.ssd_mixer_version.restype = ctypes.c_int
    lib.ssd_mixer_launch_count.argtypes = []
    lib.ssd_mixer_launch_count.restype = ctypes.c_longlong
    lib.ssd_mixer_profile_enable.argtypes = [ctypes.c_int]
    lib.ssd_mixer_profile_enable.restype = None
    lib.ssd_mixer_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                                           ctypes.POINTER(ctypes.c_int), ctypes.c_int]
    lib.ssd_mixer_profile_read.restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != SSD_OK:
        raise SsdError(status, f"{what}: {load_library().ssd_status_string(status).decode()}")


def _dev(t, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, rows: int, width: int):
    """Pointer and leading dimension of a [.., rows, width]-shaped activation view whose
    consecutive rows (tokens) are ``ld`` elements apart and whose last dim is unit-stride."""
    if t.dim() < 2 or t.shape[-1] != width:
        raise ValueError(f"{name}: expected last dim {width}, got {tuple(t.shape)}")
    if t.numel() // width != rows:
        raise ValueError(f"{name}: expected {rows} rows, got {t.numel() // width}")
    if rows == 0:          # nothing is read or written; any strides will do
        return _dev(t, name), width
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: last dim must have unit stride")
    ld = t.stride(-2)
    # all leading dims must be an even tiling by ld (token t of row i at (i*L + t) * ld)
    expect = ld
    for d in range(t.dim() - 2, -1, -1):
        if t.shape[d] > 1 and t.stride(d) != expect:
            raise ValueError(f"{name}: rows must be evenly strided")
        expect *= t.shape[d]
    return _dev(t, name), ld


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def ssd_mixer_prefill_workspace_size(dims: Dims) -> int:
    cd = dims.c()
    return int(load_library().ssd_mixer_prefill_workspace_size(ctypes.byref(cd)))


def ssd_mixer_prefill(dims: Dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                      init_ssm_state, init_conv_state, y, final_ssm_state, final_conv_state,
                      workspace, stream=None) -> None:
    lib = load_library()
    rows = dims.batch * dims.seqlen
    HP, GN = dims.d_inner, dims.ngroups * dims.dstate
    args = []
    for t, name, w in ((x, "x", HP), (z, "z", HP), (B, "B", GN), (C, "C", GN), (dt, "dt", dims.nheads)):
        args += list(_rows(t, name, rows, w))
    py, y_ld = _rows(y, "y", rows, HP)
    cd = dims.c()
    st = lib.ssd_mixer_prefill(
        ctypes.byref(cd), *args, _dev(A, "A"), _dev(D, "D"), _dev(conv_w, "conv_w"),
        _dev(conv_b, "conv_b"), _dev(dt_bias, "dt_bias"), _dev(norm_w, "norm_w"),
        _dev(init_ssm_state, "init_ssm_state"), _dev(init_conv_state, "init_conv_state"),
        py, y_ld, _dev(final_ssm_state, "final_ssm_state"), _dev(final_conv_state, "final_conv_state"),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "ssd_mixer_prefill")


def ssd_mixer_prefill_static(dims: Dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                             init_ssm_state, init_conv_state, y, final_ssm_state, final_conv_state,
                             stream=None) -> int:
    """The prefill with its scratch in the library's fixed device array (for callers that
    cannot allocate device memory); returns the C status instead of raising."""
    lib = load_library()
    rows = dims.batch * dims.seqlen
    HP, GN = dims.d_inner, dims.ngroups * dims.dstate
    args = []
    for t, name, w in ((x, "x", HP), (z, "z", HP), (B, "B", GN), (C, "C", GN), (dt, "dt", dims.nheads)):
        args += list(_rows(t, name, rows, w))
    py, y_ld = _rows(y, "y", rows, HP)
    cd = dims.c()
    return int(lib.ssd_mixer_prefill_static(
        ctypes.byref(cd), *args, _dev(A, "A"), _dev(D, "D"), _dev(conv_w, "conv_w"),
        _dev(conv_b, "conv_b"), _dev(dt_bias, "dt_bias"), _dev(norm_w, "norm_w"),
        _dev(init_ssm_state, "init_ssm_state"), _dev(init_conv_state, "init_conv_state"),
        py, y_ld, _dev(final_ssm_state, "final_ssm_state"), _dev(final_conv_state, "final_conv_state"),
        _stream(stream)))


def ssd_mixer_projection(A, W, C, workspace, stream=None) -> None:
    """C = A . W^T on the tensor cores: A [M, K], W [N, K], C [M, N], bf16 (row strides from the
    tensors; last dims unit-stride). workspace: >= 256 bytes for the status word."""
    M, K = A.shape[-2], A.shape[-1]
    N = W.shape[0]
    for t, nm in ((A, "A"), (W, "W"), (C, "C")):
        if t.dtype != torch.bfloat16 or t.stride(-1) != 1:
            raise ValueError(f"{nm}: bf16 with unit-stride rows expected")
    st = load_library().ssd_mixer_projection(M, N, K, _dev(A, "A"), A.stride(-2), _dev(W, "W"), W.stride(-2),
                                             _dev(C, "C"), C.stride(-2), _dev(workspace, "workspace"), _stream(stream))
    _check(st, "ssd_mixer_projection")


def ssd_mixer_layer_workspace_size(dims: Dims, d_model: int) -> int:
    cd = dims.c()
    return int(load_library().ssd_mixer_layer_workspace_size(ctypes.byref(cd), d_model))


def layer_prefill(dims: Dims, hidden, W_in, W_out, A, D, conv_w, conv_b, dt_bias, norm_w,
                  init_ssm_state=None, init_conv_state=None, workspace=None, out=None, norm_in_out_proj=False,
                  stream=None):
    """The whole mixer layer (in_proj, the core, out_proj) through ssd_mixer_layer_prefill.
    hidden [b, L, d_model] bf16; W_in [2HP + 2GN + H, d_model]; W_out [d_model, HP].
    norm_in_out_proj: finish a wide group's norm inside out_proj instead of in the core.
    Returns (out [b, L, d_model], final_ssm_state, final_conv_state)."""
    lib = load_library()
    d_model = hidden.shape[-1]
    rows = dims.batch * dims.seqlen
    ph, hld = _rows(hidden, "hidden", rows, d_model)
    dev = hidden.device
    if workspace is None:
        n = ssd_mixer_layer_workspace_size(dims, d_model)
        if n == 0:
            raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_mixer_layer_workspace_size: unsupported dims")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    if out is None:
        y = torch.empty(dims.batch, dims.seqlen, d_model, dtype=torch.bfloat16, device=dev)
        fs = torch.empty(dims.batch, dims.nheads, dims.headdim, dims.dstate, dtype=torch.float32, device=dev)
        fc = torch.empty(dims.batch, dims.d_inner + 2 * dims.ngroups * dims.dstate, dims.dconv - 1,
                         dtype=torch.bfloat16, device=dev)
    else:
        y, fs, fc = out
    py, yld = _rows(y, "out", rows, d_model)
    cd = dims.c()
    st = lib.ssd_mixer_layer_prefill(
        ctypes.byref(cd), d_model, ph, hld, _dev(W_in, "W_in"), _dev(W_out, "W_out"), _dev(A, "A"), _dev(D, "D"),
        _dev(conv_w, "conv_w"), _dev(conv_b, "conv_b"), _dev(dt_bias, "dt_bias"), _dev(norm_w, "norm_w"),
        _dev(init_ssm_state, "init_ssm_state"), _dev(init_conv_state, "init_conv_state"), py, yld,
        _dev(fs, "final_ssm_state"), _dev(fc, "final_conv_state"), 1 if norm_in_out_proj else 0,
        _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "ssd_mixer_layer_prefill")
    return y, fs, fc


def ssd_mixer_prefill_path(dims: Dims) -> int:
    """SSD_PATH_TENSOR_CORES, SSD_PATH_CUDA_CORES or SSD_PATH_NONE: which kernels a prefill of
    these dims runs (a host-side query)."""
    cd = dims.c()
    return int(load_library().ssd_mixer_prefill_path(ctypes.byref(cd)))


def ssd_mixer_prefill_plan(dims: Dims, sms: int = 0) -> dict:
    """How the tensor-core main kernel runs a prefill of these dims on ``sms`` SMs (0 = this
    device's): launches per call, pieces per (sequence, head) row, blocks per piece, CTAs per
    launch (a host-side query)."""
    cd = dims.c()
    out = [ctypes.c_int(0) for _ in range(4)]
    st = load_library().ssd_mixer_prefill_plan(ctypes.byref(cd), sms, *[ctypes.byref(o) for o in out])
    _check(st, "ssd_mixer_prefill_plan")
    return dict(zip(("launches", "pieces", "piece_blocks", "ctas_per_launch"), (o.value for o in out)))


def prefill_uses_tensor_cores(dims: Dims) -> bool:
    return ssd_mixer_prefill_path(dims) == SSD_PATH_TENSOR_CORES


def ssd_mixer_prefill_stage_offsets(dims: Dims) -> dict:
    """Byte offsets of xbc_act, delta and y_pre in the workspace of a CUDA-core prefill."""
    cd = dims.c()
    o = [ctypes.c_size_t(0) for _ in range(3)]
    _check(load_library().ssd_mixer_prefill_stage_offsets(ctypes.byref(cd), *[ctypes.byref(v) for v in o]),
           "ssd_mixer_prefill_stage_offsets")
    return {"xbc_act": o[0].value, "delta": o[1].value, "y_pre": o[2].value}


def ssd_mixer_prefill_static_status(stream=None) -> int:
    """Status word of the fixed array that ssd_mixer_prefill_static uses (synchronises the stream)."""
    return int(load_library().ssd_mixer_prefill_static_status(_stream(stream)))


def ssd_mixer_prefill_varlen_workspace_size(dims: Dims) -> int:
    cd = dims.c()
    return int(load_library().ssd_mixer_prefill_varlen_workspace_size(ctypes.byref(cd)))


def ssd_mixer_prefill_varlen(dims: Dims, cu_seqlens, slot_idx, has_init, x, z, B, C, dt, A, D, conv_w,
                             conv_b, dt_bias, norm_w, ssm_state, conv_state, y, workspace,
                             stream=None) -> None:
    """Packed variable-length prefill on state slots: dims.batch sequences, dims.seqlen packed
    tokens in total (x ... y are [T, width] row views); cu_seqlens int32 [b+1], slot_idx int32
    [b] or None, has_init uint8 [b] or None, all on the device."""
    lib = load_library()
    rows = dims.seqlen
    HP, GN = dims.d_inner, dims.ngroups * dims.dstate
    if cu_seqlens.dtype != torch.int32 or (slot_idx is not None and slot_idx.dtype != torch.int32):
        raise TypeError("cu_seqlens and slot_idx must be int32")
    if has_init is not None and has_init.dtype != torch.uint8:
        raise TypeError("has_init must be uint8")
    args = []
    for t, name, w in ((x, "x", HP), (z, "z", HP), (B, "B", GN), (C, "C", GN), (dt, "dt", dims.nheads)):
        args += list(_rows(t, name, rows, w))
    py, y_ld = _rows(y, "y", rows, HP)
    cd = dims.c()
    st = lib.ssd_mixer_prefill_varlen(
        ctypes.byref(cd), _dev(cu_seqlens, "cu_seqlens"), _dev(slot_idx, "slot_idx"), _dev(has_init, "has_init"),
        *args, _dev(A, "A"), _dev(D, "D"), _dev(conv_w, "conv_w"), _dev(conv_b, "conv_b"),
        _dev(dt_bias, "dt_bias"), _dev(norm_w, "norm_w"), _dev(ssm_state, "ssm_state"),
        _dev(conv_state, "conv_state"), py, y_ld, _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "ssd_mixer_prefill_varlen")


def ssd_mixer_prefill_state_workspace_size(dims: Dims) -> int:
    cd = dims.c()
    return int(load_library().ssd_mixer_prefill_state_workspace_size(ctypes.byref(cd)))


def ssd_mixer_prefill_state(dims: Dims, x, B, C, dt, A, conv_w, conv_b, dt_bias, init_ssm_state,
                            init_conv_state, final_ssm_state, final_conv_state, decay, workspace,
                            stream=None) -> None:
    """State-only prefill: final states and the per-(row, head) decay, no output rows."""
    lib = load_library()
    rows = dims.batch * dims.seqlen
    GN = dims.ngroups * dims.dstate
    args = []
    for t, name, w in ((x, "x", dims.d_inner), (B, "B", GN), (C, "C", GN), (dt, "dt", dims.nheads)):
        args += list(_rows(t, name, rows, w))
    cd = dims.c()
    st = lib.ssd_mixer_prefill_state(
        ctypes.byref(cd), *args, _dev(A, "A"), _dev(conv_w, "conv_w"), _dev(conv_b, "conv_b"),
        _dev(dt_bias, "dt_bias"), _dev(init_ssm_state, "init_ssm_state"), _dev(init_conv_state, "init_conv_state"),
        _dev(final_ssm_state, "final_ssm_state"), _dev(final_conv_state, "final_conv_state"), _dev(decay, "decay"),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "ssd_mixer_prefill_state")


def ssd_mixer_state_pass(r: int, decay, state, init, out, stream=None) -> None:
    """State entering piece r of a split sequence: decay [npieces, b, H], state
    [npieces, b, H, P, N] (zero-start final states of the pieces), init [b, H, P, N] or None."""
    b, H, P, N = out.shape
    st = load_library().ssd_mixer_state_pass(b, H, P, N, r, _dev(decay, "decay"), _dev(state, "state"),
                                             _dev(init, "init"), _dev(out, "out"), _stream(stream))
    _check(st, "ssd_mixer_state_pass")


def ssd_mixer_decode_step(dims: Dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                          ssm_state, conv_state, slot_idx, y, stream=None) -> None:
    lib = load_library()
    HP, GN = dims.d_inner, dims.ngroups * dims.dstate
    args = []
    for t, name, w in ((x, "x", HP), (z, "z", HP), (B, "B", GN), (C, "C", GN), (dt, "dt", dims.nheads)):
        args += list(_rows(t, name, dims.batch, w))
    py, y_ld = _rows(y, "y", dims.batch, HP)
    if slot_idx is not None and slot_idx.dtype != torch.int32:
        raise TypeError("slot_idx must be int32")
    cd = dims.c()
    st = lib.ssd_mixer_decode_step(
        ctypes.byref(cd), *args, _dev(A, "A"), _dev(D, "D"), _dev(conv_w, "conv_w"),
        _dev(conv_b, "conv_b"), _dev(dt_bias, "dt_bias"), _dev(norm_w, "norm_w"),
        _dev(ssm_state, "ssm_state"), _dev(conv_state, "conv_state"), _dev(slot_idx, "slot_idx"),
        py, y_ld, _stream(stream))
    _check(st, "ssd_mixer_decode_step")


def ssd_mixer_backward_workspace_size(dims: Dims) -> int:
    cd = dims.c()
    return int(load_library().ssd_mixer_backward_workspace_size(ctypes.byref(cd)))


def ssd_mixer_backward(dims: Dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                       init_ssm_state, init_conv_state, dy, dfinal_ssm_state, dfinal_conv_state,
                       dx, dz, dB, dC, ddt, dA, dD, dconv_w, dconv_b, ddt_bias, dnorm_w,
                       dinit_ssm_state, dinit_conv_state, workspace, stream=None) -> None:
    lib = load_library()
    rows = dims.batch * dims.seqlen
    HP, GN, H = dims.d_inner, dims.ngroups * dims.dstate, dims.nheads
    ins = []
    for t, name, w in ((x, "x", HP), (z, "z", HP), (B, "B", GN), (C, "C", GN), (dt, "dt", H)):
        ins += list(_rows(t, name, rows, w))
    outs = []
    for t, name, w in ((dx, "dx", HP), (dz, "dz", HP), (dB, "dB", GN), (dC, "dC", GN), (ddt, "ddt", H)):
        outs += list(_rows(t, name, rows, w))
    pdy, dy_ld = _rows(dy, "dy", rows, HP)
    cd = dims.c()
    st = lib.ssd_mixer_backward(
        ctypes.byref(cd), *ins, _dev(A, "A"), _dev(D, "D"), _dev(conv_w, "conv_w"), _dev(conv_b, "conv_b"),
        _dev(dt_bias, "dt_bias"), _dev(norm_w, "norm_w"), _dev(init_ssm_state, "init_ssm_state"),
        _dev(init_conv_state, "init_conv_state"), pdy, dy_ld, _dev(dfinal_ssm_state, "dfinal_ssm_state"),
        _dev(dfinal_conv_state, "dfinal_conv_state"), *outs, _dev(dA, "dA"), _dev(dD, "dD"),
        _dev(dconv_w, "dconv_w"), _dev(dconv_b, "dconv_b"), _dev(ddt_bias, "ddt_bias"), _dev(dnorm_w, "dnorm_w"),
        _dev(dinit_ssm_state, "dinit_ssm_state"), _dev(dinit_conv_state, "dinit_conv_state"),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "ssd_mixer_backward")


def ssd_mixer_selftest_wait(workspace, limit_cycles: int, arrive: bool, stream=None) -> None:
    st = load_library().ssd_mixer_selftest_wait(_dev(workspace, "workspace"), int(limit_cycles), int(bool(arrive)),
                                                _stream(stream))
    _check(st, "ssd_mixer_selftest_wait")


def ssd_mixer_workspace_status(workspace, stream=None) -> int:
    return int(load_library().ssd_mixer_workspace_status(_dev(workspace, "workspace"), _stream(stream)))


def alloc_workspace(dims: Dims, device="cuda") -> torch.Tensor:
    n = ssd_mixer_prefill_workspace_size(dims)
    if n == 0:
        raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_mixer_prefill_workspace_size: unsupported dims")
    return torch.empty(n, dtype=torch.uint8, device=device)


def prefill(dims: Dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
            init_ssm_state=None, init_conv_state=None, workspace=None, out=None, stream=None):
    """Allocate y, the final states and (if not given) the workspace, then run
    :func:`ssd_mixer_prefill`. Returns (y, final_ssm_state, final_conv_state)."""
    dev = x.device
    b, L, H, P, N = dims.batch, dims.seqlen, dims.nheads, dims.headdim, dims.dstate
    if out is None:
        y = torch.empty(b, L, dims.d_inner, dtype=dims.torch_dtype, device=dev)
        fs = torch.empty(b, H, P, N, dtype=torch.float32, device=dev)
        fc = torch.empty(b, dims.xbc_channels, dims.dconv - 1, dtype=dims.torch_dtype, device=dev)
    else:
        y, fs, fc = out
    ws = workspace if workspace is not None else alloc_workspace(dims, dev)
    ssd_mixer_prefill(dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                      init_ssm_state, init_conv_state, y, fs, fc, ws, stream)
    return y, fs, fc


def backward(dims: Dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w, dy,
             init_ssm_state=None, init_conv_state=None, dfinal_ssm_state=None, dfinal_conv_state=None,
             workspace=None, stream=None) -> dict:
    """Allocate the gradients and (if not given) the workspace, then run
    :func:`ssd_mixer_backward`. Returns a dict of gradients keyed like the inputs (x, z, B, C,
    dt, A, D, conv_w, conv_b, dt_bias, norm_w, init_ssm, init_conv)."""
    dev = x.device
    b, L, H, P, N, Cc = dims.batch, dims.seqlen, dims.nheads, dims.headdim, dims.dstate, dims.xbc_channels
    HP, GN, act = dims.d_inner, dims.ngroups * dims.dstate, dims.torch_dtype
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"x": torch.empty(b, L, HP, dtype=act, device=dev), "z": torch.empty(b, L, HP, dtype=act, device=dev),
         "B": torch.empty(b, L, GN, dtype=act, device=dev), "C": torch.empty(b, L, GN, dtype=act, device=dev),
         "dt": torch.empty(b, L, H, dtype=act, device=dev), "A": torch.empty(H, **f32), "D": torch.empty(H, **f32),
         "conv_w": torch.empty(Cc, dims.dconv, **f32), "conv_b": torch.empty(Cc, **f32),
         "dt_bias": torch.empty(H, **f32), "norm_w": torch.empty(HP, **f32),
         "init_ssm": torch.empty(b, H, P, N, **f32), "init_conv": torch.empty(b, Cc, dims.dconv - 1, **f32)}
    if workspace is None:
        n = ssd_mixer_backward_workspace_size(dims)
        if n == 0:
            raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_mixer_backward_workspace_size: unsupported dims")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    ssd_mixer_backward(dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w, init_ssm_state,
                       init_conv_state, dy, dfinal_ssm_state, dfinal_conv_state, g["x"], g["z"], g["B"], g["C"],
                       g["dt"], g["A"], g["D"], g["conv_w"], g["conv_b"], g["dt_bias"], g["norm_w"],
                       g["init_ssm"], g["init_conv"], workspace, stream)
    return g


def decode_step(dims: Dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                ssm_state, conv_state, slot_idx=None, y=None, stream=None):
    """Run :func:`ssd_mixer_decode_step` (states updated in place); returns y."""
    if y is None:
        y = torch.empty(dims.batch, dims.d_inner, dtype=dims.torch_dtype, device=x.device)
    ssd_mixer_decode_step(dims, x, z, B, C, dt, A, D, conv_w, conv_b, dt_bias, norm_w,
                          ssm_state, conv_state, slot_idx, y, stream)
    return y


# ------------------------------------------------------- linear attention and layer norm
def _refuse(t, name: str, dtype, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, the call on {dev}")


def _rows_on(t, name: str, rows: int, width: int, dtype, dev):
    """Pointer and row stride of `rows` evenly strided rows of `width` unit-stride elements, of the
    given type and on the given device. Dimensions of size 1 set no stride."""
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != dtype:
        _refuse(t, name, dtype, dev)
    shape = t.shape
    if not shape or shape[-1] != width or t.numel() != rows * width:
        raise ValueError(f"{name}: expected {rows} rows of {width}, got {tuple(shape)}")
    if rows == 0 or t.is_contiguous():
        return t.data_ptr(), width
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: last dim must have unit stride")
    ld, expect = width, None
    for d in range(t.dim() - 2, -1, -1):
        if shape[d] == 1:
            continue
        if expect is None:
            ld = t.stride(d)
            expect = ld * shape[d]
        elif t.stride(d) != expect:
            raise ValueError(f"{name}: rows must be evenly strided")
        else:
            expect *= shape[d]
    return t.data_ptr(), ld


def _whole(t, name: str, shape, dtype, dev):
    """Pointer of a contiguous tensor of exactly this shape, type and device (None: NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != dtype:
        _refuse(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _new_like(t):
    """A contiguous tensor of t's shape and type (empty_like keeps a dense tensor's other orders)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _device_of(t, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.device


# The handle of a device's current stream without a Stream object around it (3 us of a small call's 20).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """Makes the tensors' device current and, where a stream is given, that stream too (so that what
    the call allocates belongs to it). Yields the stream's handle."""
    __slots__ = ("dev", "stream", "ctx")

    def __init__(self, dev, stream):
        self.dev, self.stream, self.ctx = dev, stream, None

    def __enter__(self):
        dev, stream = self.dev, self.stream
        if stream is None and torch.cuda.current_device() == dev.index:
            return _raw_stream(dev.index)
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                handle = _stream(stream)     # 0, the default stream, is no external one: ExternalStream(0) is some new stream
                stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
            if stream.device != dev:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        self.ctx = [torch.cuda.device(dev)]      # entered when nothing can refuse any more
        self.ctx[0].__enter__()
        if stream is None:
            return _raw_stream(dev.index)
        self.ctx.append(torch.cuda.stream(stream))
        self.ctx[1].__enter__()
        return stream.cuda_stream

    def __exit__(self, *exc):
        while self.ctx:
            self.ctx.pop().__exit__(*exc)
        return False


def _linear_dims(dims: LinearDims) -> _CLinearDims:
    if dims.act not in _ACT_DTYPES:
        raise ValueError(f"act: expected one of {sorted(_ACT_DTYPES)}, got {dims.act!r}")
    return dims.c()


def _linear_qkv(dims: LinearDims, rows: int, q, k, v, dev):
    a, H, G = dims.torch_dtype, dims.nheads, dims.ngroups
    return (*_rows_on(q, "q", rows, H * dims.dk, a, dev), *_rows_on(k, "k", rows, G * dims.dk, a, dev),
            *_rows_on(v, "v", rows, G * dims.dv, a, dev))


def _workspace(ws, size: int, what: str, dev):
    """The given workspace's (or a new one's) pointer, bytes and tensor."""
    if ws is None:
        if size == 0:
            raise SsdError(SSD_ERR_UNSUPPORTED, f"{what}: invalid or unsupported dims")
        ws = torch.empty_strided((size,), (1,), dtype=torch.uint8, device=dev)   # less host time than torch.empty
    elif not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def ssd_mixer_linear_prefill_workspace_size(dims: LinearDims) -> int:
    return int(load_library().ssd_mixer_linear_prefill_workspace_size(ctypes.byref(_linear_dims(dims))))


def ssd_mixer_linear_prefill_varlen_workspace_size(dims: LinearDims) -> int:
    return int(load_library().ssd_mixer_linear_prefill_varlen_workspace_size(ctypes.byref(_linear_dims(dims))))


def ssd_mixer_linear_backward_workspace_size(dims: LinearDims) -> int:
    return int(load_library().ssd_mixer_linear_backward_workspace_size(ctypes.byref(_linear_dims(dims))))


def linear_prefill(dims: LinearDims, q, k, v, log_decay, init_state=None, workspace=None, out=None, stream=None):
    """Linear attention over b rows of L tokens (ssd_mixer_linear_prefill): q [b, L, H * dk], k
    [b, L, G * dk], v [b, L, G * dv], log_decay [H] fp32, init_state [b, H, dv, dk] fp32 or None.
    Returns (o [b, L, H * dv], final_state); ``out`` gives both tensors."""
    dev = _device_of(q, "q")
    cd = _linear_dims(dims)
    b, L, H = dims.batch, dims.seqlen, dims.nheads
    rows = _linear_qkv(dims, b * L, q, k, v, dev)
    sshape = (b, H, dims.dv, dims.dk)
    pd = _whole(log_decay, "log_decay", (H,), torch.float32, dev)
    pi = _whole(init_state, "init_state", sshape, torch.float32, dev)
    lib = load_library()
    with _On(dev, stream) as on:
        if out is None:
            o = q.new_empty((b, L, H * dims.dv))
            fs = log_decay.new_empty(sshape)
            po, pf = (o.data_ptr(), H * dims.dv), fs.data_ptr()
        else:
            o, fs = out
            po = _rows_on(o, "o", b * L, H * dims.dv, dims.torch_dtype, dev)
            pf = _whole(fs, "final_state", sshape, torch.float32, dev)
        pw, nw, ws = _workspace(workspace, 0 if workspace is not None else
                                lib.ssd_mixer_linear_prefill_workspace_size(ctypes.byref(cd)), "linear_prefill", dev)
        st = lib.ssd_mixer_linear_prefill(ctypes.byref(cd), *rows, pd, pi, *po, pf, pw, nw, on)
    _check(st, "ssd_mixer_linear_prefill")
    return o, fs


def linear_prefill_varlen(dims: LinearDims, cu_seqlens, slot_idx, has_init, q, k, v, log_decay, state, workspace=None,
                          o=None, stream=None):
    """Linear attention over packed sequences on state slots (ssd_mixer_linear_prefill_varlen): q
    [T, H * dk] ..., state [nslots, H, dv, dk] fp32 updated in place; cu_seqlens int32 [b + 1],
    slot_idx int32 [b] or None, has_init uint8 [b] or None. Returns o [T, H * dv]."""
    dev = _device_of(q, "q")
    cd = _linear_dims(dims)
    b, T, H = dims.batch, dims.seqlen, dims.nheads
    rows = _linear_qkv(dims, T, q, k, v, dev)
    pcu = _whole(cu_seqlens, "cu_seqlens", (b + 1,), torch.int32, dev)
    psl = _whole(slot_idx, "slot_idx", (b,), torch.int32, dev)
    phi = _whole(has_init, "has_init", (b,), torch.uint8, dev)
    pd = _whole(log_decay, "log_decay", (H,), torch.float32, dev)
    nslots = int(state.shape[0]) if isinstance(state, torch.Tensor) and state.dim() else 0
    ps = _whole(state, "state", (nslots, H, dims.dv, dims.dk), torch.float32, dev)
    lib = load_library()
    with _On(dev, stream) as on:
        if o is None:
            o = q.new_empty((T, H * dims.dv))
            po = o.data_ptr(), H * dims.dv
        else:
            po = _rows_on(o, "o", T, H * dims.dv, dims.torch_dtype, dev)
        pw, nw, ws = _workspace(workspace, 0 if workspace is not None else
                                lib.ssd_mixer_linear_prefill_varlen_workspace_size(ctypes.byref(cd)),
                                "linear_prefill_varlen", dev)
        st = lib.ssd_mixer_linear_prefill_varlen(ctypes.byref(cd), pcu, psl, phi, *rows, pd, ps, nslots, *po, pw, nw,
                                                 on)
    _check(st, "ssd_mixer_linear_prefill_varlen")
    return o


def linear_decode_step(dims: LinearDims, q, k, v, log_decay, state, slot_idx=None, o=None, stream=None):
    """One token of each of b sequences (ssd_mixer_linear_decode_step): q [b, H * dk] ..., state
    [nslots, H, dv, dk] fp32 updated in place. Returns o [b, H * dv]."""
    dev = _device_of(q, "q")
    cd = _linear_dims(dims)
    b, H = dims.batch, dims.nheads
    rows = _linear_qkv(dims, b, q, k, v, dev)
    psl = _whole(slot_idx, "slot_idx", (b,), torch.int32, dev)
    pd = _whole(log_decay, "log_decay", (H,), torch.float32, dev)
    nslots = int(state.shape[0]) if isinstance(state, torch.Tensor) and state.dim() else 0
    ps = _whole(state, "state", (nslots, H, dims.dv, dims.dk), torch.float32, dev)
    with _On(dev, stream) as on:
        if o is None:
            w = H * dims.dv
            o = torch.empty_strided((b, w), (w, 1), dtype=q.dtype, device=dev)
            po = o.data_ptr(), w
        else:
            po = _rows_on(o, "o", b, H * dims.dv, dims.torch_dtype, dev)
        st = load_library().ssd_mixer_linear_decode_step(ctypes.byref(cd), *rows, pd, ps, nslots, psl, *po, on)
    _check(st, "ssd_mixer_linear_decode_step")
    return o


def linear_backward(dims: LinearDims, q, k, v, log_decay, do, init_state=None, dfinal_state=None, workspace=None,
                    stream=None) -> dict:
    """Gradients of :func:`linear_prefill` (ssd_mixer_linear_backward) from do [b, L, H * dv] and,
    optionally, that of the final state. Returns {"q", "k", "v", "init_state"}."""
    dev = _device_of(q, "q")
    cd = _linear_dims(dims)
    b, L, H, G, a = dims.batch, dims.seqlen, dims.nheads, dims.ngroups, dims.torch_dtype
    rows = _linear_qkv(dims, b * L, q, k, v, dev)
    sshape = (b, H, dims.dv, dims.dk)
    pd = _whole(log_decay, "log_decay", (H,), torch.float32, dev)
    pi = _whole(init_state, "init_state", sshape, torch.float32, dev)
    pdo = _rows_on(do, "do", b * L, H * dims.dv, a, dev)
    pdf = _whole(dfinal_state, "dfinal_state", sshape, torch.float32, dev)
    lib = load_library()
    with _On(dev, stream) as on:
        g = {"q": q.new_empty((b, L, H * dims.dk)), "k": q.new_empty((b, L, G * dims.dk)),
             "v": q.new_empty((b, L, G * dims.dv)), "init_state": log_decay.new_empty(sshape)}
        outs = []
        for n, w in (("q", H * dims.dk), ("k", G * dims.dk), ("v", G * dims.dv)):
            outs += [g[n].data_ptr(), w]
        pw, nw, ws = _workspace(workspace, 0 if workspace is not None else
                                lib.ssd_mixer_linear_backward_workspace_size(ctypes.byref(cd)), "linear_backward", dev)
        st = lib.ssd_mixer_linear_backward(ctypes.byref(cd), *rows, pd, pi, *pdo, pdf, *outs, g["init_state"].data_ptr(),
                                           pw, nw, on)
    _check(st, "ssd_mixer_linear_backward")
    return g


def _norm_args(x, weight, groups: int):
    dev = _device_of(x, "x")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"x: expected fp32 or bf16, got {x.dtype}")
    if x.dim() < 1 or groups <= 0 or x.shape[-1] == 0 or x.shape[-1] % groups:
        raise ValueError(f"x: the last dim of {tuple(x.shape)} is not a multiple of groups = {groups}")
    C = x.shape[-1]
    rows = x.numel() // C
    return dev, C, rows, C // groups, SSD_BF16 if x.dtype == torch.bfloat16 else SSD_F32, _rows_on(x, "x", rows, C, x.dtype, dev)


def layer_norm(x, weight=None, bias=None, groups: int = 1, eps: float = 1e-5, out=None, stream=None):
    """Layer norm over each of ``groups`` contiguous runs of x's last dim (ssd_mixer_layer_norm);
    weight and bias [x.shape[-1]] fp32 or None. Returns (y, mean, rstd), the statistics fp32 of shape
    [*x.shape[:-1], groups]; ``out`` gives y (which may be x)."""
    dev, C, rows, width, act, px = _norm_args(x, weight, groups)
    pw = _whole(weight, "weight", (C,), torch.float32, dev)
    pb = _whole(bias, "bias", (C,), torch.float32, dev)
    with _On(dev, stream) as on:
        if out is None:
            y = _new_like(x)
            py = y.data_ptr(), C
        else:
            y, py = out, _rows_on(out, "out", rows, C, x.dtype, dev)
        mean = x.new_empty((*x.shape[:-1], groups), dtype=torch.float32)
        rstd = torch.empty_like(mean)
        st = load_library().ssd_mixer_layer_norm(rows, groups, width, eps, act, *px, pw, pb, *py, mean.data_ptr(),
                                                 rstd.data_ptr(), on)
    _check(st, "ssd_mixer_layer_norm")
    return y, mean, rstd


def ssd_mixer_layer_norm_backward_workspace_size(rows: int, groups: int, width: int, act: str) -> int:
    return int(load_library().ssd_mixer_layer_norm_backward_workspace_size(rows, groups, width,
                                                                          SSD_BF16 if act == "bf16" else SSD_F32))


def layer_norm_backward(dy, x, weight, mean, rstd, groups: int = 1, workspace=None, stream=None):
    """Gradients of :func:`layer_norm` (ssd_mixer_layer_norm_backward) from dy, x and the saved
    statistics. Returns (dx, dweight, dbias), the parameters' in fp32."""
    dev, C, rows, width, act, px = _norm_args(x, weight, groups)
    pdy = _rows_on(dy, "dy", rows, C, x.dtype, dev)
    pw = _whole(weight, "weight", (C,), torch.float32, dev)
    sshape = (*x.shape[:-1], groups)
    pm, pr = _whole(mean, "mean", sshape, torch.float32, dev), _whole(rstd, "rstd", sshape, torch.float32, dev)
    lib = load_library()
    with _On(dev, stream) as on:
        dx = _new_like(x)
        dweight = x.new_empty((C,), dtype=torch.float32) if weight is None else torch.empty_like(weight)
        dbias = torch.empty_like(dweight)
        pws, nws, ws = _workspace(workspace, 0 if workspace is not None else
                                  lib.ssd_mixer_layer_norm_backward_workspace_size(rows, groups, width, act),
                                  "layer_norm_backward", dev)
        st = lib.ssd_mixer_layer_norm_backward(rows, groups, width, act, *pdy, *px, pw, pm, pr, dx.data_ptr(), C,
                                               dweight.data_ptr(), dbias.data_ptr(), pws, nws, on)
    _check(st, "ssd_mixer_layer_norm_backward")
    return dx, dweight, dbias
