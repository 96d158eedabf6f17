"""Fused selective state-space scan, forward and backward, for MI355X (gfx950).

The scan itself runs in the HIP library ``libssmscan.so`` behind the C ABI of
``include/ssm_scan.h``; this package is its thin binding (``selective_scan_fwd``,
``selective_scan_bwd`` and the raw ``ssm_*`` calls), the build script and the
seeded synthetic input generators.  Beside the scan stand the operators around
it: its step for single tokens (``selective_scan_step``), the short causal
convolution (``causal_conv_fwd``, ``causal_conv_bwd``, ``causal_conv_step``) and
the layer or RMS norm (``layer_norm_fwd``, ``layer_norm_bwd``); its sibling with
one state a channel, the gated recurrence (``gated_recurrence_fwd``,
``gated_recurrence_bwd``, ``gated_recurrence_step``); and behind either the group
norm with an activation or a gate (``group_norm_fwd``, ``group_norm_bwd``).
"""
from ._binding import (EXPORTED, SSM_COMBINE_WALK, SSM_COMBINE_WAVE_SCAN, SSM_ERR_ALIAS, SSM_ERR_DEVICE_MISMATCH, SSM_ERR_HIP, SSM_ERR_INVALID_ARG,
                       SSM_ERR_NO_DEVICE, SSM_ERR_SCRATCH, SSM_ERR_UNSUPPORTED, SSM_GATE_AFTER, SSM_GATE_BEFORE,
                       SSM_GATE_NONE, SSM_IO_BF16, SSM_IO_F32, SSM_OK,
                       SSM_SCAN_NOALLOC_SCRATCH_BYTES, SsmScanError, auto_time_parts, bwd_chunk_len,
                       bwd_workspace_bytes, chunk_len, error_string, gated_chunk_len, lib, library_path, selective_scan_bwd,
                       selective_scan_fwd, ssm_conv_bwd_io, ssm_conv_dims, ssm_conv_fwd_io, ssm_conv_step_io,
                       ssm_norm_bwd_io, ssm_norm_dims, ssm_norm_fwd_io, ssm_scan_bwd_io, ssm_scan_create,
                       ssm_scan_destroy, ssm_scan_dims, ssm_scan_step_io, ssm_scan_fwd_extras, ssm_selective_scan_bwd, ssm_selective_scan_fwd, ssm_selective_scan_fwd_ex,
                       ssm_selective_scan_fwd_noalloc, workspace_bytes, ssm_gated_bwd_io, ssm_gated_dims,
                       ssm_gated_fwd_io, ssm_gated_step_io, ssm_group_norm_bwd_io, ssm_group_norm_dims,
                       ssm_group_norm_fwd_io)


_BLOCK = ("causal_conv_bwd", "causal_conv_fwd", "causal_conv_step", "gated_recurrence_bwd", "gated_recurrence_fwd",
          "gated_recurrence_step", "group_norm_bwd", "group_norm_fwd", "layer_norm_bwd", "layer_norm_fwd",
          "selective_scan_step")


def __getattr__(name):
    # their module loads on first use, and torch with their first call: the
    # package's import stays light
    if name in _BLOCK:
        from . import _block
        for k in _BLOCK:
            globals()[k] = getattr(_block, k)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


__all__ = [
    "selective_scan_step", "causal_conv_fwd", "causal_conv_bwd", "causal_conv_step", "layer_norm_fwd",
    "layer_norm_bwd", "ssm_scan_step_io", "ssm_conv_dims", "ssm_conv_fwd_io", "ssm_conv_bwd_io", "ssm_conv_step_io",
    "ssm_norm_dims", "ssm_norm_fwd_io", "ssm_norm_bwd_io",
    "gated_recurrence_fwd", "gated_recurrence_bwd", "gated_recurrence_step", "gated_chunk_len", "group_norm_fwd",
    "group_norm_bwd", "ssm_gated_dims", "ssm_gated_fwd_io", "ssm_gated_bwd_io", "ssm_gated_step_io",
    "ssm_group_norm_dims", "ssm_group_norm_fwd_io", "ssm_group_norm_bwd_io", "SSM_GATE_NONE", "SSM_GATE_AFTER",
    "SSM_GATE_BEFORE",
    "selective_scan_fwd", "ssm_scan_create", "ssm_scan_destroy", "ssm_selective_scan_fwd", "ssm_scan_dims",
    "ssm_selective_scan_fwd_ex", "ssm_scan_fwd_extras", "chunk_len", "auto_time_parts", "workspace_bytes",
    "selective_scan_bwd", "ssm_selective_scan_bwd", "ssm_scan_bwd_io", "bwd_chunk_len", "bwd_workspace_bytes",
    "SsmScanError", "error_string", "lib", "library_path", "EXPORTED", "SSM_OK", "SSM_ERR_INVALID_ARG",
    "SSM_ERR_UNSUPPORTED", "SSM_ERR_ALIAS", "SSM_ERR_HIP", "SSM_ERR_NO_DEVICE", "SSM_ERR_DEVICE_MISMATCH",
    "SSM_COMBINE_WALK", "SSM_COMBINE_WAVE_SCAN", "SSM_ERR_SCRATCH", "SSM_IO_F32", "SSM_IO_BF16", "SSM_SCAN_NOALLOC_SCRATCH_BYTES", "ssm_selective_scan_fwd_noalloc",
]
