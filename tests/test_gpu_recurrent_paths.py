"""The gated recurrence's edge cases on every kernel that a call can take, and the
group norm's narrow groups.

A call's sizes choose between workgroups that hold whole rows (16 channels, or 64
a wave) and tiles of a row on different workgroups, these in turn between 8 and 16
waves, one and two channels a lane, loads through and past the caches.  Each test
names its path and holds it against what the library's workspace tells of it, so
that another rule moves no test off its kernel unseen."""
import ctypes

import numpy as np
import pytest

import recurrent_ref as R
from block_ref import check
from test_gpu_block import DEV, Gen, _dt, bits, i32, n64, sync
from test_gpu_recurrent import (_all_ops, check_gated, check_group, gated_both, gated_inputs, group_both, group_inputs,
                                off)

pytestmark = pytest.mark.gpu

CHUNK = 64


def words(B, L, D, V, steps):
    """Bytes that tiles of `steps` steps and 64 V channels publish through."""
    chains, tiles = B * -(-D // (64 * V)), -(-L // steps)
    return 4 * (4 + 64 * V * chains * (2 * tiles + tiles // 16 + 1))


def on_path(path, io, B, L, D):
    """The call's forward takes this path: "row16", "row64", or (V, waves) of tiles; what its backward takes."""
    import selective_state_space_scan_amd as ssm
    d = ssm.ssm_gated_dims(B, L, D, ssm.SSM_IO_BF16 if io == "bf16" else ssm.SSM_IO_F32)
    fwd = ssm.lib().ssm_gated_recurrence_fwd_workspace_bytes(ctypes.byref(d))
    bwd = ssm.lib().ssm_gated_recurrence_bwd_workspace_bytes(ctypes.byref(d))
    if isinstance(path, tuple):
        of = {k for k in ((1, 8), (1, 16), (2, 8), (2, 16)) if words(B, L, D, k[0], 16 * k[1]) == fwd
              and k[0] <= -(-D // 64)}   # two channels a lane are for more than 64
        assert of == {path}, (path, of)
    else:
        assert fwd == 0 and (path == "row16") == (B * -(-D // 16) <= 512), path
    tiles = bwd == words(B, L, D, 1, 64) + 4 * -(-L // 64) * B * D
    assert tiles or bwd == (4 * B * D if B > 1 else 0)
    return "tiles" if tiles else "rows"


def same(a, b):
    """The same bits, NaNs among them."""
    import torch
    as_int = lambda t: t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)  # noqa: E731
    return (a is None and b is None) or torch.equal(as_int(a), as_int(b))


def outputs(r):
    return [*r[:3], *r[3].values()]


# path of the forward, io, B, L, D
EDGES = [
    ("row16", "f32", 5, 300, 40), ("row16", "bf16", 5, 300, 40),
    ("row64", "f32", 8, 100, 8250), ("row64", "bf16", 8, 100, 8250),          # bf16: two channels a lane
    ((1, 8), "f32", 5, 2500, 40), ((1, 8), "bf16", 5, 2500, 40),              # two spans, three backward
    ((1, 8), "f32", 3, 2500, 192), ((1, 8), "bf16", 3, 2500, 192),            # whole lines
    ((1, 16), "f32", 2, 2200, 2112), ((2, 16), "bf16", 2, 2200, 4160),
    ((2, 8), "bf16", 1, 2200, 4160), ((2, 8), "bf16", 1, 2200, 4110),         # lines that pieces share
]


def lens_of(B, L):
    return [(L, L // 2 - 10, 1, 0, 3 * L // 4, 64, L - 1, 17)[b % 8] for b in range(B)]


# ---- against 64 bits -----------------------------------------------------------

@pytest.mark.parametrize("rate", [-82.0, -30.0, -12.0, 3.0, 20.0])
@pytest.mark.parametrize("path,io,B,L,D", EDGES)
def test_decays_of_every_size(path, io, B, L, D, rate):
    """Products of decays that underflow from tile to tile, and decays whose 1 - a^2 is near fp32's smallest."""
    on_path(path, io, B, L, D)
    c = gated_inputs(io, B, L, D, 303, rate=rate)
    lens = lens_of(B, L) if B > 1 else None
    r = gated_both(c, i32(lens))
    sync()
    check_gated(io, c, lens, *r)


@pytest.mark.parametrize("path,io,B,L,D", EDGES)
def test_decays_at_their_ends(path, io, B, L, D):
    """Where 1 - a^2 is below fp32's smallest normal number it counts as 0, forward and backward: the state stays, bit
    by bit, and no input has a gradient.  An infinite exp(A_log) passes the gated input alone."""
    import torch
    on_path(path, io, B, L, D)
    c = gated_inputs(io, B, L, D, 304)
    A = torch.tensor([-float("inf"), -200.0, -104.0, -103.0, -95.0, -90.0, 0.0, 100.0, float("inf")])
    c["A"] = A.repeat(-(-D // 9))[:D].contiguous().to(DEV)
    closed = torch.arange(D, device=DEV) % 9 == 6
    c["ag"][..., closed] = -90.0
    y, last, st, g = gated_both(c)
    sync()
    keep = torch.arange(D, device=DEV) % 9 <= 6
    h0, dy, dl = c["h0"][:, keep], c["dy"][..., keep].double(), c["dl"][:, keep].double()
    assert same(y[..., keep], h0[:, None].expand(B, L, -1).to(y.dtype)) and same(last[:, keep], h0)
    assert same(st[..., keep], h0[:, None].expand(B, st.shape[1], -1))
    for k in ("dx", "dx_gate"):
        assert (g[k][..., keep] == 0).all(), k
    for k in ("da_gate", "dA_log"):   # the decay's own, -s a g h, is left: s is at most e^-90
        assert (g[k][..., keep].abs() <= 1e-30).all() and (g[k][..., closed] == 0).all(), k
    # sums of L + 1 terms in another order than the steps'
    want, mag = dl + dy.sum(1), dl.abs() + dy.abs().sum(1)
    check("dh0", n64(g["dh0"][:, keep]), n64(want), (L + 1) * R.U * n64(mag))
    x, xg = n64(c["x"][..., ~keep]), n64(c["xg"][..., ~keep])
    want = x / (1 + np.exp(-xg))
    tol = (R.sig_err(xg, io) + 8 * R.U + (2.0**-8 if io == "bf16" else 0)) * np.abs(want)
    check("y", n64(y[..., ~keep]), want, tol)
    assert (g["dA_log"][~keep] == 0).all() and (g["da_gate"][..., ~keep] == 0).all()
