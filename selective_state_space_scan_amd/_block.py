"""torch front end of the operators beside the scan in its block: the scan for
single tokens, the short causal convolution, the layer or RMS norm, the gated
recurrence and the group norm.

As for the scan, every step runs in the HIP library.  Shapes, dtypes and
devices are checked, outputs and scratch allocated and the C ABI called by the
CPython module ``_ssm_torch`` (``csrc/ssm_torch.cpp``): done here, that took up
to 8 us of a single-token call whose launch takes 4.  There is no fallback.

Like the scan's, these calls record no autograd graph: inputs that require
gradients give outputs that do not, and the ``_bwd`` calls are what a custom
``torch.autograd.Function`` is made of.  Tensors of the caller's that a call
writes (caches in place, given outputs) count as modified in place.
"""
from __future__ import annotations

import ctypes

from . import _binding as _b


def _load():
    """The marshalling module, with the HIP library's entry points bound to it."""
    import torch  # noqa: F401  the module links its libraries
    lib = _b.lib()
    try:
        from . import _ssm_torch
    except ImportError as e:
        raise ImportError("the torch marshalling module _ssm_torch is not built or does not load; run "
                          "`python -m selective_state_space_scan_amd.build` (or __graft_entry__.build())") from e
    entries = ("ssm_selective_scan_step", "ssm_causal_conv_step", "ssm_causal_conv_fwd", "ssm_causal_conv_bwd",
               "ssm_causal_conv_bwd_workspace_bytes", "ssm_layer_norm_fwd", "ssm_layer_norm_bwd",
               "ssm_layer_norm_bwd_workspace_bytes", "ssm_gated_recurrence_fwd",
               "ssm_gated_recurrence_fwd_workspace_bytes", "ssm_gated_recurrence_bwd",
               "ssm_gated_recurrence_bwd_workspace_bytes", "ssm_gated_recurrence_chunk_len",
               "ssm_gated_recurrence_step", "ssm_group_norm_fwd", "ssm_group_norm_bwd",
               "ssm_group_norm_bwd_workspace_bytes")
    _ssm_torch.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in entries), _b.handle_for,
                    _b.SsmScanError)
    return _ssm_torch


class _Unloaded:
    """Stands for the module until its first use, so that importing the package needs no built library."""

    def __getattr__(self, name):
        global _native
        _native = _load()
        return getattr(_native, name)


_native = _Unloaded()


def _on(stream, x):
    """The context of a call on ``stream``: its kernels and the memory it allocates, which the caching allocator then
    orders with them."""
    import torch
    if not torch.is_tensor(x) or x.device.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    stream = _b._stream_for(stream, x.device)
    if stream.device != x.device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {x.device}")
    return torch.cuda.stream(stream)


# ---- single tokens ---------------------------------------------------------

def selective_scan_step(x, delta, A_log, B, C, D, h, *, slots=None, h_last=None, delta_softplus: bool = True,
                        delta_clamp=None, delta_bias=None, z=None, y=None, stream=None):
    """One step of the selective scan for every row of a batch; returns y.

    x, delta: [batch, dim]; B, C: [batch, dstate]; all of one dtype
    (torch.float32 or torch.bfloat16), rows anywhere (any row stride, last
    dimension dense).  A_log [dim, dstate], D [dim] or None and delta_bias
    [dim] or None: float32.  z like x or None: output gate y * silu(z).
    delta_softplus and delta_clamp as in ``selective_scan_fwd`` (the clip
    takes a NaN to its lower bound, as there).

    h: the states, float32, [batch, dim, dstate], or with ``slots`` a cache
    [n_slots, dim, dstate] of which batch row b uses row slots[b] (int32).  A
    row whose slot lies outside the cache (-1, say) is idle: no state is touched
    and its y is 0.  Where rows name one slot, the first takes the step and the
    others are idle.  The states are updated in place, or with ``h_last`` (like
    h) written there, the rows in use only.  Asynchronous on ``stream`` (default:
    the current stream of x's device).
    """
    if stream is not None:
        with _on(stream, x):
            return selective_scan_step(x, delta, A_log, B, C, D, h, slots=slots, h_last=h_last,
                                       delta_softplus=delta_softplus, delta_clamp=delta_clamp, delta_bias=delta_bias,
                                       z=z, y=y)
    return _native.scan_step(x, delta, A_log, B, C, D, h, slots, h_last, delta_softplus, delta_clamp, delta_bias, z, y)


def causal_conv_step(x, conv, weight, bias=None, *, silu: bool = True, slots=None, conv_last=None, y=None,
                     stream=None):
    """One step of the short causal convolution for every row of a batch; returns y.

    x: [batch, dim] float32 or bfloat16, any row stride.  conv: the last
    width - 1 inputs of every row, oldest first, [batch, width - 1, dim] in x's
    dtype, or with ``slots`` a cache [n_slots, width - 1, dim]; it is moved on by
    one in place, or with ``conv_last`` (like conv) written there.  slots and
    idle rows as in ``selective_scan_step``.  weight [dim, width] (2, 3 or 4 taps)
    and bias [dim] or None: float32.  silu: y = p * sigmoid(p).
    """
    if stream is not None:
        with _on(stream, x):
            return causal_conv_step(x, conv, weight, bias, silu=silu, slots=slots, conv_last=conv_last, y=y)
    return _native.conv_step(x, conv, weight, bias, silu, slots, conv_last, y)


# ---- short causal convolution ----------------------------------------------

def causal_conv_fwd(x, weight, bias=None, valid_len=None, *, silu: bool = True, conv0=None, y=None, conv_last=None,
                    return_conv_last: bool = True, stream=None):
    """Short causal convolution of every channel, with silu; returns ``(y, conv_last)``.

    x: [batch, L, dim] float32 or bfloat16, last dimension dense, other strides
    any (one half of a projection's output, say).  weight [dim, width] (2, 3 or
    4 taps, the last on the current step) and bias [dim] or None: float32.
    valid_len [batch] int32 or None: y is 0 past it and nothing there is read.
    conv0 [batch, width - 1, dim] like x: the inputs before the first, oldest
    first (zeros if None).  conv_last, likewise: the last width - 1 inputs of
    every row, to continue from (None if return_conv_last is False and none is
    given).  Outputs are allocated unless given; y may be strided like x.
    Asynchronous on ``stream``.
    """
    if stream is not None:
        with _on(stream, x):
            return causal_conv_fwd(x, weight, bias, valid_len, silu=silu, conv0=conv0, y=y, conv_last=conv_last,
                                   return_conv_last=return_conv_last)
    return _native.conv_fwd(x, weight, bias, valid_len, silu, conv0, y, conv_last, return_conv_last)


def causal_conv_bwd(x, weight, bias, valid_len, dy, *, silu: bool = True, conv0=None, dconv_last=None, dx=None,
                    workspace=None, stream=None) -> dict:
    """Gradients of ``causal_conv_fwd`` for the loss sum(dy * y) + sum(dconv_last * conv_last).

    The forward's inputs and flags must be given again.  dy like y (any
    strides, last dimension dense); dconv_last like conv_last or None.  Returns
    a dict: dx like x (contiguous unless given, strided like x then), dweight
    [dim, width], dbias [dim] (None without bias), both float32, and dconv0
    [batch, width - 1, dim] in x's dtype (None without conv0).
    """
    if stream is not None:
        with _on(stream, x):
            return causal_conv_bwd(x, weight, bias, valid_len, dy, silu=silu, conv0=conv0, dconv_last=dconv_last,
                                   dx=dx, workspace=workspace)
    dx, dweight, dbias, dconv0 = _native.conv_bwd(x, weight, bias, valid_len, silu, conv0, dy, dconv_last, dx,
                                                  workspace)
    return dict(dx=dx, dweight=dweight, dbias=dbias, dconv0=dconv0)


# ---- norms -----------------------------------------------------------------

def layer_norm_fwd(x, weight, bias=None, valid_len=None, *, residual=None, eps: float = 1e-5, rms: bool = False,
                   y=None, residual_out=None, return_stats: bool = False, stream=None):
    """Layer norm (RMS norm with ``rms``) of x + residual over the last dimension.

    x: [rows, dim] or [batch, L, dim], float32 or bfloat16, contiguous, dim at
    most 16384.  residual like x, in x's dtype or float32, or None.  weight and
    bias (or None): [dim] float32.  valid_len [batch] int32 or None (for
    [batch, L, dim]): rows past it give 0 and are not read.

    Returns ``(y, residual_out)``, or ``(y, residual_out, mean, rstd)`` with
    ``return_stats`` (float32, what the backward takes; mean is None with rms).
    residual_out is x + residual in residual's dtype (None without residual);
    it may be given, as residual itself for an update in place, or without a
    residual to start a residual stream in its own dtype.
    """
    if stream is not None:
        with _on(stream, x):
            return layer_norm_fwd(x, weight, bias, valid_len, residual=residual, eps=eps, rms=rms, y=y,
                                  residual_out=residual_out, return_stats=return_stats)
    return _native.norm_fwd(x, weight, bias, valid_len, residual, eps, rms, y, residual_out, return_stats)


def layer_norm_bwd(dy, v, weight, mean, rstd, valid_len=None, *, dresidual_out=None, with_bias: bool = True,
                   with_residual: bool | None = None, workspace=None, stream=None) -> dict:
    """Gradients of ``layer_norm_fwd`` for the loss sum(dy * y) + sum(dresidual_out * residual_out).

    dy like y.  v: what was normalised, the forward's residual_out (or x where
    there was none).  mean and rstd: the forward's; mean None for RMS norm.
    dresidual_out like v or None.  Returns a dict: dx like dy; dresidual like v
    (the same gradient in v's dtype, and the same tensor where the dtypes are
    one; None unless ``with_residual``, which follows dresidual_out if None);
    dweight and dbias (None without ``with_bias``) [dim] float32.
    """
    if stream is not None:
        with _on(stream, dy):
            return layer_norm_bwd(dy, v, weight, mean, rstd, valid_len, dresidual_out=dresidual_out,
                                  with_bias=with_bias, with_residual=with_residual, workspace=workspace)
    dx, dresidual, dweight, dbias = _native.norm_bwd(dy, v, weight, mean, rstd, valid_len, dresidual_out, with_bias,
                                                     with_residual, workspace)
    return dict(dx=dx, dresidual=dresidual, dweight=dweight, dbias=dbias)


# ---- gated recurrence ------------------------------------------------------

def gated_recurrence_fwd(x, a_gate, x_gate, A_log, valid_len=None, *, h0=None, y=None, h_last=None,
                         return_chunk_states: bool = False, workspace=None, stream=None):
    """The gated recurrence over whole sequences; returns ``(y, h_last)``, or ``(y, h_last, chunk_states)``.

    With r = sigmoid(a_gate), i = sigmoid(x_gate) and a = exp(-exp(A_log) r), every
    channel's state is h = a h + sqrt(1 - a^2) i x, and y = h.

    x, a_gate, x_gate: [batch, L, dim] of one dtype (torch.float32 or
    torch.bfloat16), last dimension dense, other strides any (both gates may be
    halves of one projection's output).  A_log [dim] float32.  valid_len [batch]
    int32 or None: y is 0 past it, nothing there is read and the state stays.
    h0 [batch, dim] float32: the state before the first step (zeros if None);
    h_last, likewise: the state after the last valid one.  Outputs are allocated
    unless given; y may be strided like x, and h_last may be h0 itself.
    chunk_states [batch, ceil(L / gated_chunk_len()), dim] float32, what the
    backward takes: the state after every chunk.  workspace: a uint8 tensor as
    long as the library asks for (allocated if None; never shared by calls that
    may run at the same time).  Asynchronous on ``stream``.
    """
    if stream is not None:
        with _on(stream, x):
            return gated_recurrence_fwd(x, a_gate, x_gate, A_log, valid_len, h0=h0, y=y, h_last=h_last,
                                        return_chunk_states=return_chunk_states, workspace=workspace)
    return _native.gated_fwd(x, a_gate, x_gate, A_log, valid_len, h0, y, h_last, return_chunk_states, workspace)


def gated_recurrence_bwd(x, a_gate, x_gate, A_log, valid_len, dy, chunk_states, *, h0=None, dh_last=None, dx=None,
                         da_gate=None, dx_gate=None, workspace=None, stream=None) -> dict:
    """Gradients of ``gated_recurrence_fwd`` for the loss sum(dy * y) + sum(dh_last * h_last).

    The forward's inputs must be given again, with its chunk_states (None where L
    is at most ``gated_chunk_len()``).  dy like y (any strides, last dimension
    dense); dh_last like h_last or None.  Returns a dict: dx, da_gate, dx_gate like
    their inputs (contiguous unless given, strided like x then: the gates' may be
    the halves of one tensor), dA_log [dim] and dh0 like h0 (None without h0), both
    float32.
    """
    if stream is not None:
        with _on(stream, x):
            return gated_recurrence_bwd(x, a_gate, x_gate, A_log, valid_len, dy, chunk_states, h0=h0, dh_last=dh_last,
                                        dx=dx, da_gate=da_gate, dx_gate=dx_gate, workspace=workspace)
    dx, da_gate, dx_gate, dA_log, dh0 = _native.gated_bwd(x, a_gate, x_gate, A_log, valid_len, h0, dy, dh_last,
                                                          chunk_states, dx, da_gate, dx_gate, workspace)
    return dict(dx=dx, da_gate=da_gate, dx_gate=dx_gate, dA_log=dA_log, dh0=dh0)


def gated_recurrence_step(x, a_gate, x_gate, A_log, h, *, slots=None, h_last=None, y=None, stream=None):
    """One step of the gated recurrence for every row of a batch; returns y.

    x, a_gate, x_gate: [batch, dim] of one dtype, any row stride.  A_log [dim]
    float32.  h: the states, float32, [batch, dim], or with ``slots`` a cache
    [n_slots, dim]; updated in place, or with ``h_last`` (like h) written there.
    slots and idle rows as in ``selective_scan_step``.
    """
    if stream is not None:
        with _on(stream, x):
            return gated_recurrence_step(x, a_gate, x_gate, A_log, h, slots=slots, h_last=h_last, y=y)
    return _native.gated_step(x, a_gate, x_gate, A_log, h, slots, h_last, y)


# ---- group norm ------------------------------------------------------------

def group_norm_fwd(x, groups: int, weight, bias=None, valid_len=None, *, z=None, silu: bool = True,
                   gate_first: bool = False, eps: float = 1e-5, rms: bool = False, y=None, return_stats: bool = False,
                   stream=None):
    """Norm of every group of a step's channels, with an activation or a gate; returns y.

    With act(u) = u sigmoid(u) (u without ``silu``) and p the layer norm (RMS norm
    with ``rms``) of each of the ``groups`` groups of adjacent channels, by
    weight and bias: y = act(p) without z, p * act(z) with z, and with
    ``gate_first`` p of x * act(z).  Every step is normalised by itself.

    x, z (or None): [rows, dim] or [batch, L, dim], float32 or bfloat16, last
    dimension dense, other strides any; a group has at most 8192 channels.
    weight and bias (or None): [dim] float32.  valid_len [batch] int32 or None
    (for [batch, L, dim]): rows past it give 0 and are not read.  y is allocated
    unless given (strided like x).  With ``return_stats``: ``(y, mean, rstd)``, the
    statistics [..., groups] float32 that the backward takes (mean None with rms).
    """
    if stream is not None:
        with _on(stream, x):
            return group_norm_fwd(x, groups, weight, bias, valid_len, z=z, silu=silu, gate_first=gate_first, eps=eps,
                                  rms=rms, y=y, return_stats=return_stats)
    return _native.group_fwd(x, groups, weight, bias, valid_len, z, silu, gate_first, eps, rms, y, return_stats)


def group_norm_bwd(dy, x, groups: int, weight, bias, mean, rstd, valid_len=None, *, z=None, silu: bool = True,
                   gate_first: bool = False, dx=None, dz=None, workspace=None, stream=None) -> dict:
    """Gradients of ``group_norm_fwd`` for the loss sum(dy * y).

    x, z, weight, bias, valid_len and the flags: the forward's; mean and rstd as
    it returned them (mean None for RMS norm).  dy like y.  Returns a dict: dx,
    dz (None without z) like x and z (contiguous unless given, strided like x
    then); dweight and dbias (None without bias) [dim] float32.
    """
    if stream is not None:
        with _on(stream, dy):
            return group_norm_bwd(dy, x, groups, weight, bias, mean, rstd, valid_len, z=z, silu=silu,
                                  gate_first=gate_first, dx=dx, dz=dz, workspace=workspace)
    dx, dz, dweight, dbias = _native.group_bwd(dy, x, groups, weight, bias, mean, rstd, valid_len, z, silu, gate_first,
                                               dx, dz, workspace)
    return dict(dx=dx, dz=dz, dweight=dweight, dbias=dbias)
