"""MI355X-native (gfx950) Kimi Delta Attention token mixer.

The computation lives in ``libkda.so`` (C ABI declared in ``include/kda.h``,
hand-written HIP kernels); ``kda`` is its thin ctypes binding and ``synth``
draws seeded synthetic inputs.
"""
from . import synth  # noqa: F401
from .kda import (KDAError, kda_add_rmsnorm, kda_add_rmsnorm_fp8, kda_conv_prefill, kda_conv_state_bytes,  # noqa: F401
                  kda_conv_state_update, kda_conv_tree, kda_conv_tree_commit, kda_decode_step, kda_decode_tree,
                  kda_decode_tree_commit, kda_gate_prologue, kda_gemm, kda_gemm_epilogue, kda_last_error,
                  kda_output_norm_gate, kda_prefill, kda_prefill_workspace_bytes, kda_state_bytes, kda_version)
