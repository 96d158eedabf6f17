"""The operators beside the scan on the host (no GPU needed): the 64-bit
reference's gradients against central differences, and the C ABI's argument
checks, which run before anything touches the GPU (the handle's among them last,
so a NULL handle meets all others first)."""
import ctypes

import numpy as np
import pytest

import block_ref as R
import selective_state_space_scan_amd as ssm

MB = 1 << 20
INVALID, UNSUPPORTED, ALIAS = ssm.SSM_ERR_INVALID_ARG, ssm.SSM_ERR_UNSUPPORTED, ssm.SSM_ERR_ALIAS
BF16, F32 = ssm.SSM_IO_BF16, ssm.SSM_IO_F32


# ---- the reference's gradients ---------------------------------------------

def _differences(f, a, eps=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + eps
        hi = f()
        a[i] = keep - eps
        lo = f()
        a[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W,lens", [(4, [7, 2, 0]), (3, None), (2, [1, 7, 5])])
def test_conv_reference_gradients_are_its_differences(silu, W, lens):
    rng = np.random.default_rng(5 + W)
    B, L, D = 3, 7, 2
    x, w, b = rng.standard_normal((B, L, D)), rng.standard_normal((D, W)), rng.standard_normal(D)
    c0, dy = rng.standard_normal((B, W - 1, D)), rng.standard_normal((B, L, D))
    dl = rng.standard_normal((B, W - 1, D))

    def loss():
        y, last, _ = R.conv_fwd(x, w, b, lens, c0, silu)
        return float((y * dy).sum() + (last * dl).sum())

    got, _ = R.conv_bwd(x, w, b, lens, dy, c0, dl, silu)
    for name, a in (("dx", x), ("dweight", w), ("dbias", b), ("dconv0", c0)):
        d = _differences(loss, a)
        assert np.max(np.abs(got[name] - d)) <= 1e-6 * max(1.0, np.max(np.abs(d))), name


@pytest.mark.parametrize("rms", [True, False])
def test_norm_reference_gradients_are_its_differences(rms):
    rng = np.random.default_rng(8)
    x, res = rng.standard_normal((3, 6)), rng.standard_normal((3, 6)) + 0.5
    w, b = rng.standard_normal(6), rng.standard_normal(6)
    dy, dr = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))

    def loss():
        (y, v, _, _), _ = R.norm_fwd(x, w, b, res, rms=rms)
        return float((y * dy).sum() + (v * dr).sum())

    (_, v, m, r), _ = R.norm_fwd(x, w, b, res, rms=rms)
    got, _ = R.norm_bwd(dy, v, w, None if rms else m, r, dr)
    for name, a in (("dx", x), ("dresidual", res), ("dweight", w), ("dbias", b)):
        d = _differences(loss, a)
        assert np.max(np.abs(got[name] - d)) <= 1e-6 * max(1.0, np.max(np.abs(d))), name


def test_step_reference_is_the_oracle_s_last_step(oracle_mod):
    """The step's formula against the scan's oracle, one step at a time."""
    rng = np.random.default_rng(3)
    B, L, D, N = 2, 5, 16, 16
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    x, dl, Bm, Cm, z = f(B, L, D), f(B, L, D), f(B, L, N), f(B, L, N), f(B, L, D)
    A_log, Dk, bias = f(D, N) * np.float32(0.5), f(D), f(D)
    y, h = oracle_mod.selective_scan(x, dl, A_log, Bm, Cm, Dk, delta_bias=bias, z=z, delta_clamp=(0.25, 1.5))[:2]
    state = np.zeros((B, D, N))
    for t in range(L):
        yt, state, _, _ = R.scan_step(x[:, t].astype(np.float64), dl[:, t].astype(np.float64), A_log,
                                      Bm[:, t].astype(np.float64), Cm[:, t].astype(np.float64), Dk.astype(np.float64),
                                      state, bias.astype(np.float64), z[:, t].astype(np.float64), True,
                                      (0.25, 1.5))
        np.testing.assert_allclose(yt, y[:, t], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(state, h, rtol=1e-12, atol=1e-12)


# ---- argument checks ---------------------------------------------------------

def conv_dims(**kw):
    d = dict(batch=2, seqlen=8, dim=24, width=4, io_dtype=BF16, silu=1)
    d.update(kw)
    return ssm.ssm_conv_dims(*d.values())


def conv_fwd(dims=None, **kw):
    dims = conv_dims() if dims is None else dims
    io = dict(x=1 * MB, weight=2 * MB, bias=3 * MB, valid_len=4 * MB, conv0=5 * MB, y=6 * MB, conv_last=7 * MB,
              x_batch_stride=8 * 24, x_time_stride=24, y_batch_stride=8 * 24, y_time_stride=24)
    io.update(kw)
    return ssm.lib().ssm_causal_conv_fwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_conv_fwd_io(**io)), None)


def conv_bwd(dims=None, **kw):
    dims = conv_dims() if dims is None else dims
    io = dict(x=1 * MB, weight=2 * MB, bias=3 * MB, valid_len=4 * MB, conv0=5 * MB, dy=6 * MB, dconv_last=7 * MB,
              dx=8 * MB, dweight=9 * MB, dbias=10 * MB, dconv0=11 * MB, workspace=12 * MB, workspace_bytes=MB,
              x_batch_stride=8 * 24, x_time_stride=24, dy_batch_stride=8 * 24, dy_time_stride=24,
              dx_batch_stride=8 * 24, dx_time_stride=24)
    io.update(kw)
    return ssm.lib().ssm_causal_conv_bwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_conv_bwd_io(**io)), None)


def conv_step(dims=None, **kw):
    dims = conv_dims(seqlen=1) if dims is None else dims
    io = dict(x=1 * MB, weight=2 * MB, bias=3 * MB, slots=4 * MB, conv0=5 * MB, conv_last=5 * MB, y=6 * MB,
              x_row_stride=24, y_row_stride=24, n_slots=8)
    io.update(kw)
    return ssm.lib().ssm_causal_conv_step(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_conv_step_io(**io)), None)


def scan_dims(**kw):
    d = dict(batch=2, seqlen=1, dim=24, dstate=16, io_dtype=BF16, delta_softplus=1, delta_clamp=0, delta_min=0.0,
             delta_max=0.0)
    d.update(kw)
    return ssm.ssm_scan_dims(*d.values())


def scan_step(dims=None, **kw):
    dims = scan_dims() if dims is None else dims
    io = dict(x=1 * MB, delta=2 * MB, A_log=3 * MB, B=4 * MB, C=5 * MB, D=6 * MB, delta_bias=7 * MB, z=8 * MB,
              slots=9 * MB, h0=10 * MB, h_last=10 * MB, y=11 * MB, x_row_stride=24, delta_row_stride=24,
              B_row_stride=16, C_row_stride=16, z_row_stride=24, y_row_stride=24, n_slots=8)
    io.update(kw)
    return ssm.lib().ssm_selective_scan_step(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_scan_step_io(**io)), None)


def norm_dims(**kw):
    d = dict(batch=2, seqlen=8, dim=24, io_dtype=BF16, residual_dtype=F32, rms=0, eps=1e-5)
    d.update(kw)
    return ssm.ssm_norm_dims(*d.values())


def norm_fwd(dims=None, **kw):
    dims = norm_dims() if dims is None else dims
    io = dict(x=1 * MB, residual=2 * MB, weight=3 * MB, bias=4 * MB, valid_len=5 * MB, y=6 * MB, residual_out=7 * MB,
              mean=8 * MB, rstd=9 * MB)
    io.update(kw)
    return ssm.lib().ssm_layer_norm_fwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_norm_fwd_io(**io)), None)


def norm_bwd(dims=None, **kw):
    dims = norm_dims() if dims is None else dims
    io = dict(dy=1 * MB, v=2 * MB, weight=3 * MB, mean=4 * MB, rstd=5 * MB, valid_len=6 * MB, dresidual_out=7 * MB,
              dx=8 * MB, dresidual=9 * MB, dweight=10 * MB, dbias=11 * MB, workspace=12 * MB, workspace_bytes=MB)
    io.update(kw)
    return ssm.lib().ssm_layer_norm_bwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_norm_bwd_io(**io)), None)


CALLS = dict(conv_fwd=conv_fwd, conv_bwd=conv_bwd, conv_step=conv_step, scan_step=scan_step, norm_fwd=norm_fwd,
             norm_bwd=norm_bwd)
# A misaligned input fails after every check of sizes, strides and required
# pointers and before those of overlap, so it tells an accepted call (-2) from a
# refused one (-1) although both meet the NULL handle's -1 in the end.
ODD = dict(conv_fwd=dict(weight=2 * MB + 2), conv_bwd=dict(weight=2 * MB + 2), conv_step=dict(weight=2 * MB + 2),
           scan_step=dict(A_log=3 * MB + 2), norm_fwd=dict(weight=3 * MB + 2), norm_bwd=dict(weight=3 * MB + 2))


@pytest.mark.parametrize("op", CALLS)
def test_valid_arguments_reach_the_handle_check(op):
    assert CALLS[op]() == INVALID
    assert CALLS[op](**ODD[op]) == UNSUPPORTED


@pytest.mark.parametrize("op", CALLS)
def test_null_dims_or_io(op):
    f = getattr(ssm.lib(), {"conv_fwd": "ssm_causal_conv_fwd", "conv_bwd": "ssm_causal_conv_bwd",
                            "conv_step": "ssm_causal_conv_step", "scan_step": "ssm_selective_scan_step",
                            "norm_fwd": "ssm_layer_norm_fwd", "norm_bwd": "ssm_layer_norm_bwd"}[op])
    dims = {"conv_fwd": conv_dims(), "conv_bwd": conv_dims(), "conv_step": conv_dims(seqlen=1),
            "scan_step": scan_dims(), "norm_fwd": norm_dims(), "norm_bwd": norm_dims()}[op]
    assert f(None, None, None, None) == INVALID
    assert f(None, ctypes.byref(dims), None, None) == INVALID


OPTIONAL = dict(conv_fwd=("bias", "valid_len", "conv0", "conv_last"),
                conv_bwd=("bias", "valid_len", "conv0", "dconv_last", "dbias", "dconv0"),
                conv_step=("bias", "slots"), scan_step=("D", "delta_bias", "z", "slots"),
                norm_fwd=("residual", "residual_out", "bias", "valid_len", "mean", "rstd"),
                norm_bwd=("valid_len", "dresidual_out", "dresidual", "dbias"))
REQUIRED = dict(conv_fwd=("x", "weight", "y"), conv_bwd=("x", "weight", "dy", "dx", "dweight", "workspace"),
                conv_step=("x", "weight", "conv0", "conv_last", "y"),
                scan_step=("x", "delta", "A_log", "B", "C", "h0", "h_last", "y"), norm_fwd=("x", "weight", "y"),
                norm_bwd=("dy", "v", "weight", "mean", "rstd", "dx", "dweight", "workspace"))


@pytest.mark.parametrize("op", CALLS)
def test_required_and_optional_pointers(op):
    for name in OPTIONAL[op]:
        assert CALLS[op](**{name: None, **ODD[op]}) == UNSUPPORTED, name
    for name in REQUIRED[op]:
        assert CALLS[op](**{**ODD[op], name: None}) == INVALID, name
    for name in OPTIONAL[op] + REQUIRED[op]:
        assert CALLS[op](**{name: 60 * MB + 1}) == UNSUPPORTED, name


@pytest.mark.parametrize("op", ["conv_fwd", "conv_bwd", "conv_step"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(dim=-1), INVALID), (dict(io_dtype=2), INVALID), (dict(silu=2), INVALID),
    (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(dim=2**29), UNSUPPORTED),
    (dict(batch=2**31), UNSUPPORTED)])
def test_conv_dims(op, kw, code):
    base = dict(seqlen=1) if op == "conv_step" else {}
    assert CALLS[op](conv_dims(**base, **kw)) == code
    assert ssm.lib().ssm_causal_conv_bwd_workspace_bytes(ctypes.byref(conv_dims(**kw))) == -1


def test_conv_lengths():
    assert conv_fwd(conv_dims(seqlen=-1)) == INVALID and conv_bwd(conv_dims(seqlen=-1)) == INVALID
    assert conv_step(conv_dims(seqlen=2)) == INVALID and conv_step(conv_dims(seqlen=0)) == INVALID
    assert conv_fwd(conv_dims(seqlen=2**31)) == UNSUPPORTED
    # no steps need no x, y, dy, dx
    none = dict(x=None, y=None)
    assert conv_fwd(conv_dims(seqlen=0), **none, weight=2 * MB + 2) == UNSUPPORTED
    assert ssm.lib().ssm_causal_conv_bwd_workspace_bytes(None) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(dim=-1), INVALID), (dict(io_dtype=2), INVALID), (dict(delta_softplus=2), INVALID),
    (dict(seqlen=2), INVALID), (dict(delta_clamp=2), INVALID),
    (dict(delta_clamp=1, delta_min=0.5, delta_max=0.1), INVALID), (dict(delta_clamp=1, delta_min=-1.0), INVALID),
    (dict(delta_clamp=1, delta_max=float("inf")), INVALID), (dict(delta_clamp=1, delta_max=float("nan")), INVALID),
    (dict(dstate=8), UNSUPPORTED), (dict(dstate=48), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED)])
def test_scan_step_dims(kw, code):
    assert scan_step(scan_dims(**kw)) == code


@pytest.mark.parametrize("op", ["norm_fwd", "norm_bwd"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(dim=-1), INVALID), (dict(io_dtype=2), INVALID),
    (dict(residual_dtype=2), INVALID), (dict(io_dtype=F32, residual_dtype=BF16), INVALID), (dict(rms=2), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(dim=16385), UNSUPPORTED), (dict(batch=2**31), UNSUPPORTED),
    (dict(batch=2**30, seqlen=2**30), UNSUPPORTED)])
def test_norm_dims(op, kw, code):
    assert CALLS[op](norm_dims(**kw)) == code
    assert ssm.lib().ssm_layer_norm_bwd_workspace_bytes(ctypes.byref(norm_dims(**kw))) == -1


def test_rms_needs_no_mean():
    assert norm_bwd(norm_dims(rms=1), mean=None, **ODD["norm_bwd"]) == UNSUPPORTED


def test_workspaces():
    need = ssm.lib().ssm_causal_conv_bwd_workspace_bytes(ctypes.byref(conv_dims()))
    assert need > 0
    assert conv_bwd(workspace_bytes=need, **ODD["conv_bwd"]) == UNSUPPORTED
    assert conv_bwd(workspace_bytes=need - 4, **ODD["conv_bwd"]) == INVALID
    assert conv_bwd(workspace_bytes=-1, **ODD["conv_bwd"]) == INVALID
    need = ssm.lib().ssm_layer_norm_bwd_workspace_bytes(ctypes.byref(norm_dims()))
    assert need > 0
    assert norm_bwd(workspace_bytes=need, **ODD["norm_bwd"]) == UNSUPPORTED
    assert norm_bwd(workspace_bytes=need - 4, **ODD["norm_bwd"]) == INVALID
    assert norm_bwd(workspace_bytes=-1, **ODD["norm_bwd"]) == INVALID


@pytest.mark.parametrize("batch,seqlen,dim,width", [(4096, 8, 2048, 4), (65536, 2, 1024, 4), (3, 0, 24, 2),
                                                    (512, 52, 1024, 3)])
def test_conv_workspace_of_short_rows(batch, seqlen, dim, width):
    """One set of sums a row where a row's steps are one workgroup's, as the header says."""
    d = conv_dims(batch=batch, seqlen=seqlen, dim=dim, width=width)
    assert ssm.lib().ssm_causal_conv_bwd_workspace_bytes(ctypes.byref(d)) == batch * (width + 1) * dim * 4


def test_strides():
    bad = ODD["conv_fwd"]
    assert conv_fwd(x_time_stride=-24, **bad) == INVALID and conv_fwd(y_batch_stride=-1, **bad) == INVALID
    assert conv_fwd(x_time_stride=0, x_batch_stride=0, **bad) == UNSUPPORTED  # a repeated input may be read
    assert conv_fwd(y_time_stride=23, **bad) == INVALID          # steps of y overlap
    assert conv_fwd(y_batch_stride=8 * 24 - 1, **bad) == INVALID  # rows of y overlap
    assert conv_fwd(y_batch_stride=24, y_time_stride=48, **bad) == UNSUPPORTED  # time-major: rows within a step
    assert conv_fwd(y_batch_stride=24, y_time_stride=47, **bad) == INVALID
    assert conv_fwd(x_time_stride=2**62, **bad) == INVALID       # the span leaves 62 bits
    bad = ODD["conv_bwd"]
    assert conv_bwd(dx_time_stride=0, **bad) == INVALID and conv_bwd(dy_time_stride=0, **bad) == UNSUPPORTED
    assert conv_bwd(dy_time_stride=-1, **bad) == INVALID
    for f, bad, names in ((conv_step, ODD["conv_step"], ("x",)),
                          (scan_step, ODD["scan_step"], ("x", "delta", "B", "C", "z"))):
        for k in names:
            assert f(**{k + "_row_stride": -1}, **bad) == INVALID and f(**{k + "_row_stride": 0}, **bad) == UNSUPPORTED
        assert f(y_row_stride=23, **bad) == INVALID and f(n_slots=-1, **bad) == INVALID
        assert f(n_slots=0, **bad) == UNSUPPORTED  # every row is idle
        assert f(n_slots=2**31, **bad) == UNSUPPORTED


@pytest.mark.parametrize("op", CALLS)
def test_outputs_overlap_nothing(op):
    outs = dict(conv_fwd=("y", "conv_last"), conv_bwd=("dx", "dweight", "dbias", "dconv0", "workspace"),
                conv_step=("y",), scan_step=("y",), norm_fwd=("y", "residual_out", "mean", "rstd"),
                norm_bwd=("dx", "dresidual", "dweight", "dbias", "workspace"))[op]
    for o in outs:
        for other in OPTIONAL[op] + REQUIRED[op]:
            if other == o or (op, o, other) == ("norm_fwd", "residual_out", "residual"):
                continue
            assert CALLS[op](**{o: 50 * MB, other: 50 * MB}) == ALIAS, (o, other)


def test_caches_in_place_only_as_a_whole():
    assert conv_step(conv0=5 * MB, conv_last=5 * MB) == INVALID     # the handle
    assert conv_step(conv0=5 * MB, conv_last=5 * MB + 2) == ALIAS
    assert scan_step(h0=10 * MB, h_last=10 * MB) == INVALID
    assert scan_step(h0=10 * MB, h_last=10 * MB + 64) == ALIAS
    assert norm_fwd(residual=2 * MB, residual_out=2 * MB) == INVALID
    assert norm_fwd(residual=2 * MB, residual_out=2 * MB + 4) == ALIAS


def test_empty_batches_need_only_the_handle():
    none = {k: None for k in OPTIONAL["conv_fwd"] + REQUIRED["conv_fwd"]}
    assert conv_fwd(conv_dims(batch=0), **none) == INVALID
    none = {k: None for k in OPTIONAL["scan_step"] + REQUIRED["scan_step"]}
    assert scan_step(scan_dims(batch=0), **none) == INVALID
    none = {k: None for k in OPTIONAL["norm_fwd"] + REQUIRED["norm_fwd"]}
    assert norm_fwd(norm_dims(batch=0), **none) == INVALID


def test_norm_rows_of_no_elements():
    """dim 0 needs no rows and no weight; misaligned statistics are looked at all the same, so they are not skipped."""
    none = {k: None for k in OPTIONAL["norm_fwd"] + REQUIRED["norm_fwd"]}
    assert norm_fwd(norm_dims(dim=0), **none) == INVALID   # the handle
    assert norm_fwd(norm_dims(dim=0), **{**none, "rstd": 9 * MB + 2}) == UNSUPPORTED
    assert norm_fwd(norm_dims(dim=0), **{**none, "mean": 9 * MB, "rstd": 9 * MB}) == ALIAS


def test_binding_rejects_cpu_tensors():
    import torch
    x = torch.zeros(2, 16)
    for f in (lambda: ssm.selective_scan_step(x, x, torch.zeros(16, 16), x, x, None, torch.zeros(2, 16, 16)),
              lambda: ssm.causal_conv_step(x, torch.zeros(2, 3, 16), torch.zeros(16, 4)),
              lambda: ssm.causal_conv_fwd(x[None], torch.zeros(16, 4)),
              lambda: ssm.causal_conv_bwd(x[None], torch.zeros(16, 4), None, None, x[None]),
              lambda: ssm.layer_norm_fwd(x, torch.zeros(16)),
              lambda: ssm.layer_norm_bwd(x, x, torch.zeros(16), None, torch.zeros(2))):
        with pytest.raises(ValueError):
            f()


def test_marshalling_module_is_built_and_refuses_plainly():
    """The CPython module loads, and what is no tensor, or too few arguments, is a Python exception."""
    import torch
    from selective_state_space_scan_amd import _block
    from selective_state_space_scan_amd import build as B
    import os
    assert os.path.exists(B.TORCH_LIB_PATH), "run __graft_entry__.build() first"
    n = _block._load()
    with pytest.raises(TypeError):
        n.scan_step()
    with pytest.raises(TypeError):
        n.conv_step(1, 2, 3, None, True, None, None, None)
    with pytest.raises(ValueError):
        n.conv_step(torch.zeros(2, 16), torch.zeros(2, 3, 16), torch.zeros(16, 4), None, True, None, None, None)
    with pytest.raises(TypeError):
        n.bind(1, 2)


def test_marshalling_module_is_host_code():
    """Compiled by the host compiler against torch's headers; no GPU source in it."""
    from selective_state_space_scan_amd import build as B
    cmd = B.torch_command("/tmp/x.so")
    assert cmd[0] == "g++" and cmd[cmd.index("-o") + 1] == "/tmp/x.so" and B.TORCH_SRC in cmd
    assert "-lc10_hip" in cmd and "-ltorch_python" in cmd and not any("offload-arch" in a for a in cmd)
