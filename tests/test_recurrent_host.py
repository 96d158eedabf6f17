"""The gated recurrence and the group norm on the host (no GPU needed): the 64-bit
reference against central differences and against itself piece by piece, and the
C ABI's argument checks, which run before anything touches the GPU (the handle's
among them last, so a NULL handle meets all others first)."""
import ctypes

import numpy as np
import pytest

import recurrent_ref as R
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


def _same(got, d, name):
    assert np.max(np.abs(got - d)) <= 1e-6 * max(1.0, np.max(np.abs(d))), name


@pytest.mark.parametrize("lens", [[7, 2, 0], None])
def test_recurrence_reference_gradients_are_its_differences(lens):
    rng = np.random.default_rng(31)
    B, L, D = 3, 7, 2
    x, ag, xg, dy = (rng.standard_normal((B, L, D)) for _ in range(4))
    A, h0, dl = rng.standard_normal(D) - 1, rng.standard_normal((B, D)), rng.standard_normal((B, D))

    def loss():
        (y, last, _), _ = R.gated_fwd(x, ag, xg, A, lens, h0)
        return float((y * dy).sum() + (last * dl).sum())

    got, _ = R.gated_bwd(x, ag, xg, A, lens, dy, h0, dl)
    for name, a in (("dx", x), ("da_gate", ag), ("dx_gate", xg), ("dA_log", A), ("dh0", h0)):
        _same(got[name], _differences(loss, a), name)


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("gate", ["none", "after", "before"])
def test_group_norm_reference_gradients_are_its_differences(gate, silu, rms):
    rng = np.random.default_rng(32)
    x, dy, z = (rng.standard_normal((3, 6)) for _ in range(3))
    w, b = rng.standard_normal(6), rng.standard_normal(6)
    z = None if gate == "none" else z
    kw = dict(z=z, silu=silu, gate_first=gate == "before")

    def loss():
        (y, _, _), _ = R.group_fwd(x, 2, w, b, rms=rms, **kw)
        return float((y * dy).sum())

    (_, m, r), _ = R.group_fwd(x, 2, w, b, rms=rms, **kw)
    got, _ = R.group_bwd(dy, x, 2, w, b, None if rms else m, r, **kw)
    for name, a in (("dx", x), ("dz", z), ("dweight", w), ("dbias", b)):
        if a is not None:
            _same(got[name], _differences(loss, a), name)


def test_one_group_is_the_layer_norm():
    import block_ref
    rng = np.random.default_rng(33)
    x, w, b = rng.standard_normal((4, 10)), rng.standard_normal(10), rng.standard_normal(10)
    (y, m, r), _ = R.group_fwd(x, 1, w, b, silu=False)
    (ly, _, lm, lr), _ = block_ref.norm_fwd(x, w, b)
    for got, want in ((y, ly), (m[:, 0], lm), (r[:, 0], lr)):
        np.testing.assert_allclose(got, want, rtol=1e-13, atol=1e-13)


def test_decays_keep_the_state_s_variance():
    """sqrt(1 - a^2): independent inputs of variance 1 behind an open gate keep the state's variance at 1."""
    rng = np.random.default_rng(34)
    B, L, D = 400, 60, 4
    x = rng.standard_normal((B, L, D))
    (y, last, _), _ = R.gated_fwd(x, np.zeros((B, L, D)), np.full((B, L, D), 40.0), np.array([-3.0, -2, -1, 0]), None,
                                  rng.standard_normal((B, D)))
    # 1600 values: the estimate's standard error is sqrt(2 / 1600) = 0.035
    assert abs(last.var() - 1) < 5 * 0.036


# ---- argument checks ---------------------------------------------------------

def gated_dims(**kw):
    d = dict(batch=2, seqlen=80, dim=24, io_dtype=BF16)
    d.update(kw)
    return ssm.ssm_gated_dims(*d.values())


_S = dict(batch_stride=80 * 24, time_stride=24)


def _strides(*names):
    return {f"{n}_{k}": v for n in names for k, v in _S.items()}


def gated_fwd(dims=None, **kw):
    dims = gated_dims() if dims is None else dims
    io = dict(x=1 * MB, a_gate=2 * MB, x_gate=3 * MB, A_log=4 * MB, valid_len=5 * MB, h0=6 * MB, y=7 * MB, h_last=8 * MB,
              chunk_states=9 * MB, workspace=10 * MB, workspace_bytes=MB, **_strides("x", "a_gate", "x_gate", "y"))
    io.update(kw)
    return ssm.lib().ssm_gated_recurrence_fwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_gated_fwd_io(**io)), None)


def gated_bwd(dims=None, **kw):
    dims = gated_dims() if dims is None else dims
    io = dict(x=1 * MB, a_gate=2 * MB, x_gate=3 * MB, A_log=4 * MB, valid_len=5 * MB, h0=6 * MB, dy=7 * MB,
              dh_last=8 * MB, chunk_states=9 * MB, dx=10 * MB, da_gate=11 * MB, dx_gate=12 * MB, dA_log=13 * MB,
              dh0=14 * MB, workspace=15 * MB, workspace_bytes=MB,
              **_strides("x", "a_gate", "x_gate", "dy", "dx", "da_gate", "dx_gate"))
    io.update(kw)
    return ssm.lib().ssm_gated_recurrence_bwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_gated_bwd_io(**io)), None)


def gated_step(dims=None, **kw):
    dims = gated_dims(seqlen=1) if dims is None else dims
    io = dict(x=1 * MB, a_gate=2 * MB, x_gate=3 * MB, A_log=4 * MB, slots=5 * MB, h0=6 * MB, h_last=6 * MB, y=7 * MB,
              x_row_stride=24, a_gate_row_stride=24, x_gate_row_stride=24, y_row_stride=24, n_slots=8)
    io.update(kw)
    return ssm.lib().ssm_gated_recurrence_step(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_gated_step_io(**io)), None)


def group_dims(**kw):
    d = dict(batch=2, seqlen=80, dim=24, groups=3, io_dtype=BF16, rms=0, silu=1, gate=ssm.SSM_GATE_AFTER, eps=1e-5)
    d.update(kw)
    return ssm.ssm_group_norm_dims(*d.values())


def group_fwd(dims=None, **kw):
    dims = group_dims() if dims is None else dims
    io = dict(x=1 * MB, z=2 * MB, weight=3 * MB, bias=4 * MB, valid_len=5 * MB, y=6 * MB, mean=7 * MB, rstd=8 * MB,
              **_strides("x", "z", "y"))
    io.update(kw)
    return ssm.lib().ssm_group_norm_fwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_group_norm_fwd_io(**io)), None)


def group_bwd(dims=None, **kw):
    dims = group_dims() if dims is None else dims
    io = dict(dy=1 * MB, x=2 * MB, z=3 * MB, weight=4 * MB, bias=5 * MB, mean=6 * MB, rstd=7 * MB, valid_len=8 * MB,
              dx=9 * MB, dz=10 * MB, dweight=11 * MB, dbias=12 * MB, workspace=13 * MB, workspace_bytes=MB,
              **_strides("dy", "x", "z", "dx", "dz"))
    io.update(kw)
    return ssm.lib().ssm_group_norm_bwd(None, ctypes.byref(dims), ctypes.byref(ssm.ssm_group_norm_bwd_io(**io)), None)


CALLS = dict(gated_fwd=gated_fwd, gated_bwd=gated_bwd, gated_step=gated_step, group_fwd=group_fwd, group_bwd=group_bwd)
ENTRY = dict(gated_fwd="ssm_gated_recurrence_fwd", gated_bwd="ssm_gated_recurrence_bwd",
             gated_step="ssm_gated_recurrence_step", group_fwd="ssm_group_norm_fwd", group_bwd="ssm_group_norm_bwd")
DIMS = dict(gated_fwd=gated_dims, gated_bwd=gated_dims, gated_step=lambda **kw: gated_dims(**{"seqlen": 1, **kw}),
            group_fwd=group_dims, group_bwd=group_dims)
# A misaligned input fails after every check of sizes, strides and required
# pointers and before those of overlap, so it tells an accepted call (-2) from a
# refused one (-1) although both meet the NULL handle's -1 in the end.
ODD = dict(gated_fwd=dict(A_log=4 * MB + 2), gated_bwd=dict(A_log=4 * MB + 2), gated_step=dict(A_log=4 * MB + 2),
           group_fwd=dict(weight=3 * MB + 2), group_bwd=dict(weight=4 * MB + 2))
OPTIONAL = dict(gated_fwd=("valid_len", "h0", "h_last", "chunk_states"), gated_bwd=("valid_len", "h0", "dh_last", "dh0"),
                gated_step=("slots",), group_fwd=("bias", "valid_len", "mean", "rstd"),
                group_bwd=("bias", "valid_len", "dbias"))
REQUIRED = dict(gated_fwd=("x", "a_gate", "x_gate", "A_log", "y"),
                gated_bwd=("x", "a_gate", "x_gate", "A_log", "dy", "chunk_states", "dx", "da_gate", "dx_gate", "dA_log",
                           "workspace"),
                gated_step=("x", "a_gate", "x_gate", "A_log", "h0", "h_last", "y"),
                group_fwd=("x", "z", "weight", "y"),
                group_bwd=("dy", "x", "z", "weight", "mean", "rstd", "dx", "dz", "dweight", "workspace"))


@pytest.mark.parametrize("op", CALLS)
def test_valid_arguments_reach_the_handle_check(op):
    assert CALLS[op]() == INVALID
    assert CALLS[op](**ODD[op]) == UNSUPPORTED


@pytest.mark.parametrize("op", CALLS)
def test_null_dims_or_io(op):
    f = getattr(ssm.lib(), ENTRY[op])
    assert f(None, None, None, None) == INVALID
    assert f(None, ctypes.byref(DIMS[op]()), None, None) == INVALID


@pytest.mark.parametrize("op", CALLS)
def test_required_and_optional_pointers(op):
    for name in OPTIONAL[op]:
        assert CALLS[op](**{**ODD[op], name: None}) == UNSUPPORTED, name
    for name in REQUIRED[op]:
        assert CALLS[op](**{**ODD[op], name: None}) == INVALID, name
    for name in OPTIONAL[op] + REQUIRED[op]:
        assert CALLS[op](**{name: 60 * MB + 1}) == UNSUPPORTED, name


@pytest.mark.parametrize("op", ["gated_fwd", "gated_bwd", "gated_step"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(dim=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(io_dtype=2), INVALID),
    (dict(dim=2**29), UNSUPPORTED), (dict(batch=2**31), UNSUPPORTED), (dict(seqlen=2**31), UNSUPPORTED),
    (dict(batch=2**30, seqlen=2**30), UNSUPPORTED)])
def test_gated_dims(op, kw, code):
    assert CALLS[op](DIMS[op](**kw)) == code
    for f in ("fwd", "bwd"):
        need = getattr(ssm.lib(), f"ssm_gated_recurrence_{f}_workspace_bytes")
        assert need(ctypes.byref(gated_dims(**kw))) == -1 and need(None) == -1


def test_step_limits():
    assert gated_step(gated_dims(seqlen=2)) == INVALID and gated_step(gated_dims(seqlen=0)) == INVALID
    assert gated_step(gated_dims(seqlen=1, batch=65536), **ODD["gated_step"]) == UNSUPPORTED
    bad = ODD["gated_step"]
    assert gated_step(n_slots=-1, **bad) == INVALID and gated_step(n_slots=2**31, **bad) == UNSUPPORTED
    assert gated_step(n_slots=0, h0=None, h_last=None, **bad) == UNSUPPORTED  # every row is idle


@pytest.mark.parametrize("op", ["group_fwd", "group_bwd"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(dim=-1), INVALID), (dict(io_dtype=2), INVALID),
    (dict(groups=0), INVALID), (dict(groups=-3), INVALID), (dict(groups=5), INVALID), (dict(groups=48), INVALID),
    (dict(rms=2), INVALID), (dict(silu=2), INVALID), (dict(gate=3), INVALID), (dict(gate=-1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(dim=8193, groups=1), UNSUPPORTED),
    (dict(dim=2**29, groups=2**29), UNSUPPORTED), (dict(batch=2**31), UNSUPPORTED),
    (dict(batch=2**16, seqlen=2**16), UNSUPPORTED)])
def test_group_dims(op, kw, code):
    assert CALLS[op](group_dims(**kw)) == code
    assert ssm.lib().ssm_group_norm_bwd_workspace_bytes(ctypes.byref(group_dims(**kw))) == -1
    assert ssm.lib().ssm_group_norm_bwd_workspace_bytes(None) == -1


def test_gate_and_z_go_together():
    none = group_dims(gate=ssm.SSM_GATE_NONE)
    assert group_fwd(none, **ODD["group_fwd"]) == INVALID and group_fwd(none, z=None, **ODD["group_fwd"]) == UNSUPPORTED
    bad = ODD["group_bwd"]
    assert group_bwd(none, **bad) == INVALID and group_bwd(none, z=None, **bad) == INVALID
    assert group_bwd(none, z=None, dz=None, **bad) == UNSUPPORTED
    # strides of a z that is not there are not looked at
    assert group_fwd(none, z=None, z_time_stride=-1, **ODD["group_fwd"]) == UNSUPPORTED
    for gate in (ssm.SSM_GATE_AFTER, ssm.SSM_GATE_BEFORE):
        assert group_fwd(group_dims(gate=gate), z=None, **ODD["group_fwd"]) == INVALID


def test_rms_needs_no_mean():
    assert group_bwd(group_dims(rms=1), mean=None, **ODD["group_bwd"]) == UNSUPPORTED


# Sizes at a limit, behind pointers so far apart that nothing overlaps: a call whose sizes are taken meets the NULL
# handle (-1), the others -2.
def far(op, dims, **kw):
    n = dims.seqlen * dims.dim
    names = dict(gated_fwd=("x", "a_gate", "x_gate", "y"), group_fwd=("x", "z", "y"), group_bwd=("dy", "x", "z", "dx", "dz"),
                 gated_bwd=("x", "a_gate", "x_gate", "dy", "dx", "da_gate", "dx_gate"), gated_step=())[op]
    io = {k: (i + 1) << 42 for i, k in enumerate(OPTIONAL[op] + REQUIRED[op] + ("workspace",))}
    for k in names:
        io.update({k + "_batch_stride": n, k + "_time_stride": dims.dim})
    if "workspace" not in REQUIRED[op] + (("workspace",) if op == "gated_fwd" else ()):
        del io["workspace"]
    else:
        io["workspace_bytes"] = 1 << 41
    return CALLS[op](dims, **{**io, **kw})


def test_columns_of_the_sums_fit_their_grid():
    """A weight's gradient is summed by 1024 work-items for 16 columns, and a launch counts them in 32 bits."""
    most = 2**26 - 16
    for kw in (dict(batch=2, seqlen=1), dict(batch=1, seqlen=129)):
        for dim, code in ((most, INVALID), (most + 1, UNSUPPORTED), (2**29 - 1, UNSUPPORTED)):
            assert far("gated_bwd", gated_dims(dim=dim, **kw)) == code, (dim, kw)
    # one short row has its sums without a second pass
    assert far("gated_bwd", gated_dims(batch=1, seqlen=128, dim=most + 16)) == INVALID
    for dim, dbias, code in ((most, None, INVALID), (most + 1, None, UNSUPPORTED), (most // 2, 1 << 52, INVALID),
                             (most // 2 + 1, 1 << 52, UNSUPPORTED), (2**29 - 1, None, UNSUPPORTED)):
        d = group_dims(batch=1, seqlen=1, dim=dim, groups=dim)
        assert far("group_bwd", d, dbias=dbias) == code, (dim, dbias)
    # sums over nothing take another pass
    assert far("gated_bwd", gated_dims(batch=0, dim=most + 1)) == INVALID
    assert far("group_bwd", group_dims(batch=0, dim=most + 1, groups=1 + most)) == INVALID


def test_tiles_and_the_words_between_them_fit_their_grids():
    """Rows cut into tiles: a work-item clears four of the words that tiles publish, 64 or 128 channels of them also
    where a row has one."""
    for op, L, words in (("gated_fwd", 257, lambda B: 4 + 64 * B * 5),      # two tiles a row
                         ("gated_bwd", 129, lambda B: 4 + 64 * B * 7)):     # three
        most = max(B for B in range(2**34 // (words(1) - 4) - 8, 2**34 // (words(1) - 4) + 8)
                   if (words(B) // 4 + 255) // 256 * 256 < 2**32)
        for B, code in ((most, INVALID), (most + 1, UNSUPPORTED), (most * 2, UNSUPPORTED), (2**31 - 1, UNSUPPORTED)):
            d = gated_dims(batch=B, seqlen=L, dim=1)
            got = far(op, d, **{k: 0 for k in ("x_batch_stride", "a_gate_batch_stride", "x_gate_batch_stride")})
            assert got == code, (op, B)
    # whole rows: a workgroup each, and its work-items
    for op in ("gated_fwd", "gated_bwd"):
        for B, L, code in ((2**26 - 1, 2, INVALID), (2**26, 2, UNSUPPORTED), (2**31 - 1, 1, UNSUPPORTED),
                           (2**22 - 1, 128, INVALID), (2**22, 128, INVALID if op == "gated_fwd" else UNSUPPORTED)):
            assert far(op, gated_dims(batch=B, seqlen=L, dim=1)) == code, (op, B, L)


def test_states_of_no_steps_fit_their_grid():
    """Without steps the state, or its gradient, is copied by a work-item an element."""
    for op in ("gated_fwd", "gated_bwd"):
        for dim, code in ((2**22 - 256, INVALID), (2**22, UNSUPPORTED)):
            assert far(op, gated_dims(batch=2**10, seqlen=0, dim=dim)) == code, (op, dim)
    # nothing to copy
    big = gated_dims(batch=2**10, seqlen=0, dim=2**22)
    assert far("gated_fwd", big, h_last=None) == INVALID and far("gated_fwd", big, h0=1 << 50, h_last=1 << 50) == INVALID
    assert far("gated_bwd", big, dh0=None) == INVALID


def test_one_short_row_takes_no_scratch_backward():
    """Its sums are its gradient."""
    need = ssm.lib().ssm_gated_recurrence_bwd_workspace_bytes
    for L, dim in ((1, 1), (80, 24), (512, 64), (128, 9000), (0, 24)):
        assert need(ctypes.byref(gated_dims(batch=1, seqlen=L, dim=dim))) == 0, (L, dim)
    for B, L, dim in ((2, 80, 24), (1, 513, 64), (1, 129, 9000)):
        assert need(ctypes.byref(gated_dims(batch=B, seqlen=L, dim=dim))) >= 4 * B * dim, (B, L, dim)
    one = gated_dims(batch=1)
    assert gated_bwd(one, workspace=None, workspace_bytes=0, **ODD["gated_bwd"]) == UNSUPPORTED
    assert gated_bwd(one, workspace=None, workspace_bytes=0) == INVALID                   # the handle
    assert gated_bwd(one, workspace=15 * MB + 4) == UNSUPPORTED                           # what is given is looked at
    assert gated_bwd(one, workspace=1 * MB) == ALIAS


def test_short_sequences_need_no_kept_states():
    n = ssm.gated_chunk_len()
    assert n == 64
    assert gated_bwd(gated_dims(seqlen=n), chunk_states=None, **ODD["gated_bwd"]) == UNSUPPORTED
    assert gated_bwd(gated_dims(seqlen=n + 1), chunk_states=None, **ODD["gated_bwd"]) == INVALID


def test_workspaces():
    for op, name, dims in (("gated_bwd", "gated_recurrence_bwd", gated_dims()), ("group_bwd", "group_norm_bwd", group_dims())):
        need = getattr(ssm.lib(), f"ssm_{name}_workspace_bytes")(ctypes.byref(dims))
        assert need > 0
        assert CALLS[op](workspace_bytes=need, **ODD[op]) == UNSUPPORTED
        assert CALLS[op](workspace_bytes=need - 4, **ODD[op]) == INVALID
        assert CALLS[op](workspace_bytes=-1, **ODD[op]) == INVALID
    assert gated_fwd(workspace_bytes=-1, **ODD["gated_fwd"]) == INVALID
    d = gated_dims(batch=4, seqlen=16384, dim=1024)
    need = ssm.lib().ssm_gated_recurrence_fwd_workspace_bytes(ctypes.byref(d))
    assert need >= 0
    far = {k: v << 40 for k, v in dict(x=1, a_gate=2, x_gate=3, y=4).items()}
    far.update({f"{k}_batch_stride": 16384 * 1024 for k in ("x", "a_gate", "x_gate", "y")})
    far.update({f"{k}_time_stride": 1024 for k in ("x", "a_gate", "x_gate", "y")})
    assert gated_fwd(d, workspace=None, workspace_bytes=0, **far, **ODD["gated_fwd"]) == (INVALID if need else UNSUPPORTED)
    # a call that is too small for a workspace takes none
    assert gated_fwd(gated_dims(seqlen=1), workspace=None, workspace_bytes=0, **ODD["gated_fwd"]) == UNSUPPORTED


@pytest.mark.parametrize("op,ins,outs", [
    ("gated_fwd", ("x", "a_gate", "x_gate"), ("y",)),
    ("gated_bwd", ("x", "a_gate", "x_gate", "dy"), ("dx", "da_gate", "dx_gate")),
    ("group_fwd", ("x", "z"), ("y",)), ("group_bwd", ("x", "z", "dy"), ("dx", "dz"))])
def test_strides(op, ins, outs):
    f, bad = CALLS[op], ODD[op]
    for k in ins + outs:
        assert f(**{k + "_time_stride": -24}, **bad) == INVALID and f(**{k + "_batch_stride": -1}, **bad) == INVALID
        assert f(**{k + "_time_stride": 2**62}, **bad) == INVALID       # the span leaves 62 bits
    for k in ins:
        assert f(**{k + "_time_stride": 0, k + "_batch_stride": 0}, **bad) == UNSUPPORTED  # a repeated input may be read
    for k in outs:
        assert f(**{k + "_time_stride": 23}, **bad) == INVALID             # steps overlap
        assert f(**{k + "_batch_stride": 80 * 24 - 1}, **bad) == INVALID   # rows overlap
        assert f(**{k + "_batch_stride": 24, k + "_time_stride": 48}, **bad) == UNSUPPORTED  # time-major
        assert f(**{k + "_batch_stride": 24, k + "_time_stride": 47}, **bad) == INVALID


def test_step_strides():
    bad = ODD["gated_step"]
    for k in ("x", "a_gate", "x_gate"):
        assert gated_step(**{k + "_row_stride": -1}, **bad) == INVALID
        assert gated_step(**{k + "_row_stride": 0}, **bad) == UNSUPPORTED
    assert gated_step(y_row_stride=23, **bad) == INVALID


@pytest.mark.parametrize("op", CALLS)
def test_outputs_overlap_nothing(op):
    outs = dict(gated_fwd=("y", "h_last", "chunk_states", "workspace"),
                gated_bwd=("dx", "da_gate", "dx_gate", "dA_log", "dh0", "workspace"), gated_step=("y",),
                group_fwd=("y", "mean", "rstd"), group_bwd=("dx", "dz", "dweight", "dbias", "workspace"))[op]
    for o in outs:
        for other in OPTIONAL[op] + REQUIRED[op] + (("workspace",) if op == "gated_fwd" else ()):
            if other == o or (op, {o, other}) == ("gated_fwd", {"h_last", "h0"}):
                continue
            assert CALLS[op](**{o: 50 * MB, other: 50 * MB}) == ALIAS, (o, other)


def test_columns_of_one_buffer_do_not_overlap():
    """Both gates' gradients in one [batch, L, 2 dim] buffer, its other half another input: ranges that interleave."""
    wide = dict(da_gate_batch_stride=80 * 48, da_gate_time_stride=48, dx_gate_batch_stride=80 * 48, dx_gate_time_stride=48)
    at = lambda off: dict(da_gate=50 * MB, dx_gate=50 * MB + off * 2, **wide)  # noqa: E731
    assert gated_bwd(**at(24)) == INVALID                       # the handle: accepted
    assert gated_bwd(**at(23)) == ALIAS and gated_bwd(**at(25)) == ALIAS and gated_bwd(**at(0)) == ALIAS
    assert gated_bwd(**at(24 + 48 * 3)) == INVALID and gated_bwd(**at(24 + 48 * 3 - 1)) == ALIAS
    assert gated_bwd(da_gate=50 * MB + 48, dx_gate=50 * MB, **wide) == INVALID
    # strides that are no multiples of one another are taken as ranges
    assert gated_bwd(**{**at(24), "dx_gate_time_stride": 49, "dx_gate_batch_stride": 80 * 49}) == ALIAS
    # x read from one half, y written to the other
    two = dict(x_batch_stride=80 * 48, x_time_stride=48, y_batch_stride=80 * 48, y_time_stride=48)
    assert gated_fwd(x=50 * MB, y=50 * MB + 48, **two) == INVALID and gated_fwd(x=50 * MB, y=50 * MB + 46, **two) == ALIAS
    assert group_fwd(x=50 * MB, y=50 * MB + 48, **two) == INVALID and group_fwd(x=50 * MB, y=50 * MB, **two) == ALIAS
    # time-major: a batch row's columns within a step
    tm = dict(x_batch_stride=48, x_time_stride=96, y_batch_stride=48, y_time_stride=96)
    assert gated_fwd(x=50 * MB, y=50 * MB + 48, **tm) == INVALID and gated_fwd(x=50 * MB, y=50 * MB + 96, **tm) == ALIAS
    # a single row each has no stride
    one = gated_dims(batch=1, seqlen=1)
    assert gated_fwd(one, x=50 * MB, y=50 * MB + 48) == INVALID and gated_fwd(one, x=50 * MB, y=50 * MB + 46) == ALIAS


def test_states_in_place_only_as_a_whole():
    assert gated_fwd(h0=6 * MB, h_last=6 * MB) == INVALID     # the handle
    assert gated_fwd(h0=6 * MB, h_last=6 * MB + 4) == ALIAS
    assert gated_step(h0=6 * MB, h_last=6 * MB + 64) == ALIAS


def test_empty_batches_need_only_the_handle():
    for op, kw in (("gated_fwd", {}), ("gated_step", dict(seqlen=1)), ("group_fwd", {})):
        none = {k: None for k in OPTIONAL[op] + REQUIRED[op]}
        assert CALLS[op](DIMS[op](batch=0, **kw), **none) == INVALID
        assert CALLS[op](DIMS[op](dim=0, **kw), **none) == INVALID
    # no steps: sums over nothing and the states alone
    none = {k: None for k in REQUIRED["gated_fwd"]}
    assert gated_fwd(gated_dims(seqlen=0), **none, h0=6 * MB + 2) == UNSUPPORTED
    none = {k: None for k in REQUIRED["gated_bwd"] if k != "dA_log"}
    assert gated_bwd(gated_dims(seqlen=0), **none, h0=6 * MB + 2) == UNSUPPORTED
    assert gated_bwd(gated_dims(seqlen=0), **{**none, "dA_log": None}) == INVALID


def test_group_norm_rows_of_no_elements():
    none = {k: None for k in OPTIONAL["group_fwd"] + REQUIRED["group_fwd"]}
    assert group_fwd(group_dims(dim=0), **{**none, "rstd": 9 * MB + 2}) == UNSUPPORTED
    assert group_fwd(group_dims(dim=0), **{**none, "mean": 9 * MB, "rstd": 9 * MB}) == ALIAS


def test_binding_rejects_cpu_tensors_and_what_is_none():
    import torch
    x, A = torch.zeros(2, 3, 16), torch.zeros(16)
    for f in (lambda: ssm.gated_recurrence_fwd(x, x, x, A),
              lambda: ssm.gated_recurrence_bwd(x, x, x, A, None, x, None),
              lambda: ssm.gated_recurrence_step(x[0], x[0], x[0], A, torch.zeros(3, 16)),
              lambda: ssm.group_norm_fwd(x, 2, A),
              lambda: ssm.group_norm_bwd(x, x, 2, A, None, None, torch.zeros(2, 3, 2)),
              lambda: ssm.group_norm_fwd(x, 2, A, stream=7)):
        with pytest.raises(ValueError):
            f()
    from selective_state_space_scan_amd import _block
    n = _block._load()
    for name in ("gated_fwd", "gated_bwd", "gated_step", "group_fwd", "group_bwd"):
        with pytest.raises(TypeError):
            getattr(n, name)()
    with pytest.raises(TypeError):
        n.gated_step(1, 2, 3, None, None, None, None, None)
