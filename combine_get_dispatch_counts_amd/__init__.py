"""MI355X-native single-GPU hot path of DeepEP-style MoE dispatch / combine.

The work runs in hand-written HIP kernels for gfx950 behind the C ABI of
``libepx.so`` (include/epx.h); this package is the torch binding. Every call
loads the library first and raises ImportError if it has not been built --
there is no fallback implementation. (Importing the package itself does not
need the library, so ``python -m combine_get_dispatch_counts_amd.build`` can
run before it exists.)
"""
from ._lib import EpxError

from .api import (  # noqa: E402
    Balance,
    Dispatched,
    Layout,
    LowLatency,
    Normed,
    alloc_balance,
    alloc_dispatch,
    alloc_layout,
    alloc_ll,
    alloc_norm,
    balance_loss,
    balance_workspace,
    calibrate_sweep_rate,
    combine,
    combine_backward,
    combine_final,
    combine_partial,
    dispatch,
    dispatch_fused,
    fused_launches,
    fused_workspace_size,
    get_dispatch_layout,
    get_dispatch_layout_noalloc,
    get_error,
    get_sweep_rate,
    grouped_gemm,
    grouped_swiglu,
    ll_dispatch,
    ll_grouped_gemm,
    ll_grouped_swiglu,
    ll_reset,
    ll_size_hint,
    moe_decode,
    moe_decode_workspace,
    quantize_weights,
    Received,
    recv_permute,
    rms_norm,
    rms_norm_backward,
    rms_norm_backward_workspace,
    route,
    route_backward,
    scale_stride,
    set_sweep_rate,
    workspace_size,
)

__all__ = ["EpxError", "Layout", "Dispatched", "LowLatency", "workspace_size", "ll_size_hint",
           "scale_stride", "get_error", "alloc_layout", "get_dispatch_layout",
           "get_dispatch_layout_noalloc", "alloc_dispatch",
           "dispatch", "combine", "combine_partial", "combine_final", "ll_reset", "alloc_ll",
           "ll_dispatch", "Received", "recv_permute", "fused_workspace_size",
           "fused_launches", "dispatch_fused", "set_sweep_rate", "get_sweep_rate",
           "calibrate_sweep_rate", "quantize_weights", "grouped_gemm", "grouped_swiglu",
           "ll_grouped_gemm", "ll_grouped_swiglu", "moe_decode_workspace", "moe_decode", "Normed",
           "alloc_norm", "rms_norm", "rms_norm_backward_workspace", "rms_norm_backward", "route",
           "Balance", "alloc_balance", "balance_workspace", "balance_loss", "route_backward",
           "combine_backward"]
