"""B200 (sm_100a) CUDA library for the Mamba-2 SSD mixer core of Nemotron-H hybrids, with
linear attention with a decay per head and layer norm beside it.

The compute lives in ``libssd_mixer.so`` (C ABI: include/ssd_mixer.h). This package
holds the kernels' sources (csrc/), the build script, the ctypes binding
(:mod:`.ssd_mixer`) and the seeded synthetic workloads (:mod:`.workloads`).
Importing the package does not load the library; the first call does.
"""
from .ssd_mixer import (Dims, LinearDims, SsdError, alloc_workspace, backward, decode_step, layer_norm,  # noqa: F401
                        layer_norm_backward, linear_backward, linear_decode_step, linear_prefill,
                        linear_prefill_varlen, load_library, prefill,
                        ssd_mixer_backward, ssd_mixer_backward_workspace_size, ssd_mixer_decode_step,
                        ssd_mixer_prefill, ssd_mixer_prefill_state, ssd_mixer_prefill_varlen,
                        ssd_mixer_prefill_workspace_size, ssd_mixer_state_pass, ssd_mixer_workspace_status)
