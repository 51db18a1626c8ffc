"""B200-native Kimi Delta Attention (KDA) operator.

``chunk_fwd`` (chunked prefill), ``chunk_bwd`` (its backward pass) and
``recurrent_step`` (batched decode) run
hand-written sm_100a CUDA kernels through the library's C ABI
(``include/kda.h``), and so do the layer operators around the recurrence:
``short_conv_fwd`` / ``_step`` / ``_bwd``, ``ssm_scan_fwd`` / ``ssm_step`` /
``ssm_scan_bwd`` and ``group_norm_fwd`` / ``_bwd``.  The binding only marshals arguments; there is no CPU
fallback: on a machine without the built library or a CUDA device the calls
raise.
"""
from .binding import (  # noqa: F401
    KDAError,
    chunk_bwd,
    chunk_bwd_workspace_bytes,
    chunk_fwd,
    chunk_fwd_workspace_bytes,
    chunk_transition,
    state_affine,
    recurrent_step,
    load_library,
    library_path,
)
from .layers import (  # noqa: F401
    group_norm_bwd,
    group_norm_fwd,
    group_norm_workspace_bytes,
    short_conv_bwd,
    short_conv_bwd_workspace_bytes,
    short_conv_fwd,
    short_conv_step,
    ssm_scan_bwd,
    ssm_scan_bwd_workspace_bytes,
    ssm_scan_fwd,
    ssm_scan_fwd_workspace_bytes,
    ssm_step,
)

__all__ = ["chunk_fwd", "chunk_bwd", "recurrent_step", "chunk_transition", "state_affine",
           "chunk_fwd_workspace_bytes",
           "chunk_bwd_workspace_bytes", "short_conv_fwd", "short_conv_step", "short_conv_bwd",
           "short_conv_bwd_workspace_bytes", "ssm_scan_fwd", "ssm_step", "ssm_scan_bwd",
           "ssm_scan_fwd_workspace_bytes", "ssm_scan_bwd_workspace_bytes", "group_norm_fwd",
           "group_norm_bwd", "group_norm_workspace_bytes", "KDAError", "load_library", "library_path"]
