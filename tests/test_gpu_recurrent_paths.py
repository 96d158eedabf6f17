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

@pytest.mark.parametrize("path,io,B,L,D,lens", [
    ((2, 16), "bf16", 2, 2200, 4160, [2200, 1300]),      # what training takes, whole lines
    ((2, 16), "bf16", 1, 4400, 4160, None),              # two spans
    ((2, 8), "bf16", 1, 2200, 4160, [2177]),
    ((1, 16), "f32", 1, 4400, 2112, None),
    ((1, 16), "f32", 2, 2200, 2112, [1990, 2200]),
    ((1, 16), "bf16", 64, 2100, 64, [2100 - 31 * b for b in range(64)]),
    ((1, 8), "bf16", 3, 2500, 192, [2500, 0, 2433]),
    ((1, 8), "f32", 3, 2500, 192, None),
    ((2, 16), "bf16", 2, 2101, 8256, [2101, 700]),       # backward tiles dealt in pairs
    ((1, 16), "f32", 1, 2101, 16448, None),
])
def test_tiles_of_whole_lines(path, io, B, L, D, lens):
    """Rows whose pieces are whole lines of 128 bytes, read past the caches; run to run the same bits, and the state
    in place."""
    import selective_state_space_scan_amd as ssm
    assert on_path(path, io, B, L, D) == "tiles"
    c = gated_inputs(io, B, L, D, 301, wide=B == 2)
    assert all(c[k].data_ptr() % 128 == 0 and c[k].stride(1) * c[k].element_size() % 128 == 0 for k in ("x", "ag", "xg", "dy"))
    one, two = gated_both(c, i32(lens)), gated_both(c, i32(lens))
    sync()
    assert all(same(a, b) for a, b in zip(outputs(one), outputs(two)))
    h = c["h0"].clone()
    y, last = ssm.gated_recurrence_fwd(c["x"], c["ag"], c["xg"], c["A"], i32(lens), h0=h, h_last=h)[:2]
    assert same(y, one[0]) and same(last, one[1]) and last is h
    check_gated(io, c, lens, *one)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L,lens", [(1, None), (9, [8]), (100, None), (128, [128]), (128, [0])])
def test_one_short_row_of_many_channels(io, L, lens):
    """A row that 64-channel workgroups hold: its sums are dA_log, without scratch."""
    D = 8250
    assert on_path("row64", io, 1, L, D) == "rows"
    c = gated_inputs(io, 1, L, D, 302)
    r = gated_both(c, i32(lens))
    sync()
    check_gated(io, c, lens, *r)


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


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_lengths_around_every_edge_of_tiles_and_spans(io):
    lens = sorted({n + d for n in (0, 16, 64, 128, 256, 1024, 1088, 2048, 2112, 2176) for d in (-1, 0, 1) if n + d >= 0})
    B, L, D = len(lens), 2200, 5
    assert on_path((1, 8), io, B, L, D) == "tiles"
    c = gated_inputs(io, B, L, D, 305)
    r = gated_both(c, i32(lens))
    sync()
    check_gated(io, c, lens, *r)


@pytest.mark.parametrize("path,io,B,L,D", [e for e in EDGES if isinstance(e[0], tuple)])
def test_in_pieces(path, io, B, L, D):
    """A sequence cut anywhere and carried on, the state updated in place, is the whole sequence within its counted
    error."""
    import torch
    import selective_state_space_scan_amd as ssm
    on_path(path, io, B, L, D)
    c = gated_inputs(io, B, L, D, 306)
    lens = lens_of(B, L)
    (ry, rl, _), (ty, tl, _) = R.gated_fwd(n64(c["x"]), n64(c["ag"]), n64(c["xg"]), n64(c["A"]), lens, n64(c["h0"]), io)
    for cut in (1, 64, 1100, L - 1):
        h = c["h0"].clone()
        ys = []
        for part in (slice(0, cut), slice(cut, L)):
            vl = i32([min(max(n - part.start, 0), part.stop - part.start) for n in lens])
            before = h.clone()
            ys.append(ssm.gated_recurrence_fwd(c["x"][:, part], c["ag"][:, part], c["xg"][:, part], c["A"], vl, h0=h,
                                               h_last=h)[0])
            assert all(same(h[b], before[b]) for b in range(B) if int(vl[b]) == 0)
        sync()
        check("y", n64(torch.cat(ys, 1)), ry, ty)
        check("h_last", n64(h), rl, tl)


# ---- bit by bit ----------------------------------------------------------------

@pytest.mark.parametrize("path,io,B,L,D", EDGES)
def test_padding_reaches_nothing(path, io, B, L, D):
    """NaN, infinities and the type's lowest value past a row's end change no bit."""
    import torch
    on_path(path, io, B, L, D)
    lens = lens_of(B, L) if B > 1 else [L // 2 - 10]
    c = gated_inputs(io, B, L, D, 307)
    want = outputs(gated_both(c, i32(lens)))
    for b, n in enumerate(lens):
        for t in (want[0], *want[3:6]):
            assert not bits(t[b, n:]).any()   # +0
    for bad in (float("nan"), float("inf"), torch.finfo(_dt(io)).min):
        k = {n: t.clone() for n, t in c.items()}
        for b, n in enumerate(lens):
            for name in ("x", "ag", "xg", "dy"):
                k[name][b, n:] = bad
        assert all(same(a, b) for a, b in zip(outputs(gated_both(k, i32(lens))), want))


@pytest.mark.parametrize("path,io,B,L,D", EDGES)
def test_bad_values_stay_in_their_channel_and_row(path, io, B, L, D):
    """NaNs, among them the one whose bits are all ones, which tiles never publish as it is, and infinities."""
    import torch
    on_path(path, io, B, L, D)
    c = gated_inputs(io, B, L, D, 308)
    good = outputs(gated_both(c))
    at, cols = L // 2, (7, D - 1)
    ok = torch.ones(D, dtype=torch.bool, device=DEV)
    ok[list(cols)] = False
    for name, value in [(n, v) for n in ("x", "ag", "xg", "dy", "h0", "dl") for v in ("nan", "ones")] + [
            ("x", "inf"), ("h0", "inf")]:
        k = {n: t.clone() for n, t in c.items()}
        t = k[name]
        where = t[0] if name in ("h0", "dl") else t[0, at]
        if value == "ones":
            where.view(torch.int32 if t.dtype == torch.float32 else torch.int16)[list(cols)] = -1
        else:
            where[list(cols)] = float(value)
        r = outputs(gated_both(k))
        for i, (a, b) in enumerate(zip(r, good)):
            assert same(a[..., ok], b[..., ok]), (name, value, i)
            if i != 6:   # dA_log has no rows
                assert same(a[1:], b[1:]), (name, value, i)
        y, dx = r[0][0][:, list(cols)], r[3][0][:, list(cols)]
        first = 0 if name == "h0" else at
        if name in ("x", "ag", "xg", "h0"):   # the state forgets none of them, and knows nothing of them before they come
            assert (torch.isposinf(y[first:]) if value == "inf" else torch.isnan(y[first:])).all(), (name, value)
            assert same(y[:first], good[0][0, :first][:, list(cols)]), (name, value)
        if name in ("dy", "dl"):
            assert torch.isnan(dx[:at + 1]).all() and same(y, good[0][0][:, list(cols)]), (name, value)


@pytest.mark.parametrize("offset", [1, 3])
@pytest.mark.parametrize("path,io,B,L,D", EDGES)
def test_unaligned_views(path, io, B, L, D, offset):
    on_path(path, io, B, L, D)
    c = gated_inputs(io, B, L, D, 309)
    o = {k: off(t, offset) for k, t in c.items()}
    dx = off(c["x"], offset)
    assert all(same(a, b) for a, b in zip(outputs(gated_both(c)), outputs(gated_both(o, dx=dx))))


@pytest.mark.parametrize("path,io,B,L,D", EDGES)
def test_time_major_and_repeated_inputs(path, io, B, L, D):
    """Tensors as [L, B, D] buffers seen as [B, L, D]; inputs with stride 0."""
    import torch
    import selective_state_space_scan_amd as ssm
    on_path(path, io, B, L, D)
    c = gated_inputs(io, B, L, D, 310)
    tm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    want = outputs(gated_both(c))
    m = {k: tm(t) if t.dim() == 3 else t for k, t in c.items()}
    assert all(same(a, b) for a, b in zip(outputs(gated_both(m, dx=tm(torch.zeros_like(c["x"])))), want))
    y = tm(torch.zeros_like(c["x"]))
    got = ssm.gated_recurrence_fwd(m["x"], m["ag"], m["xg"], m["A"], h0=m["h0"], y=y)
    assert got[0] is y and same(y, want[0]) and same(got[1], want[1])
    r = dict(c, x=c["x"][:1].expand(B, L, D), ag=c["ag"][:, :1].expand(B, L, D), dy=c["dy"][:1, :1].expand(B, L, D))
    s = {k: t.contiguous() for k, t in r.items()}
    assert all(same(a, b) for a, b in zip(outputs(gated_both(r)), outputs(gated_both(s))))


def test_streams_of_tiles():
    """Tiles on another stream, and on two at once."""
    import torch
    assert on_path((1, 8), "bf16", 3, 2500, 136) == "tiles"
    sets = [_all_ops(311, 2500), _all_ops(321, 2500)]
    want = [{k: [t.clone() for t in f()] for k, f in ops} for ops in sets]
    sync()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for name, f in sets[0]:
        for how in (streams[0], streams[0].cuda_stream):
            got = f(how)
            streams[0].synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[0][name])), name
    got = [{}, {}]
    for _ in range(5):
        for i in (0, 1):
            for name, f in sets[i]:
                got[i][name] = f(streams[i])
    sync()
    for i in (0, 1):
        for name in want[i]:
            assert all(torch.equal(a, b) for a, b in zip(got[i][name], want[i][name])), (i, name)


# ---- limits --------------------------------------------------------------------

def test_the_most_columns_that_are_summed():
    """The backward's widest calls: their last columns are those of a call on them alone; one more is refused."""
    import torch
    import selective_state_space_scan_amd as ssm
    D, n = 2**26 - 16, 48
    x = torch.empty((1, 1, D), dtype=torch.bfloat16, device=DEV)
    x.view(torch.int16).random_(0x3f00, 0x3fff)   # 0.5 to 2
    A = torch.linspace(-5, 1, D, device=DEV)
    two = x.expand(2, 1, D)
    g = ssm.gated_recurrence_bwd(two, two, two, A, None, two, None)
    last = two[..., D - n:]
    r = ssm.gated_recurrence_bwd(last, last, last, A[D - n:], None, last, None)
    for k in ("dx", "da_gate", "dx_gate", "dA_log"):
        assert same(g[k][..., D - n:], r[k]), k
    ssm.gated_recurrence_bwd(x, x, x, A, None, x, None)   # one row: no second pass
    del g
    G = D // 16
    y, m, s = ssm.group_norm_fwd(x, G, A, return_stats=True)
    g = ssm.group_norm_bwd(x, x, G, A, None, m, s)
    last = x[..., D - n:]
    r = ssm.group_norm_bwd(last, last, n // 16, A[D - n:], None, m[..., G - n // 16:].contiguous(),
                           s[..., G - n // 16:].contiguous())
    assert same(g["dx"][..., D - n:], r["dx"]) and same(g["dweight"][D - n:], r["dweight"])
    wide = torch.ones((2, 1, 1), dtype=torch.bfloat16, device=DEV).expand(2, 1, D + 16).contiguous()
    w, st = torch.ones(D + 16, device=DEV), torch.ones((2, 1, G + 1), device=DEV)
    for f in (lambda: ssm.gated_recurrence_bwd(wide, wide, wide, w, None, wide, None),
              lambda: ssm.group_norm_bwd(wide, wide, G + 1, w, None, st, st),
              lambda: ssm.group_norm_bwd(x, x, G, A, A, m, s)):   # the bias's sums beside the weight's
        with pytest.raises(ssm.SsmScanError) as e:
            f()
        assert e.value.code == ssm.SSM_ERR_UNSUPPORTED


# ---- narrow groups ---------------------------------------------------------------

@pytest.mark.parametrize("gate", ["none", "after", "before"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 7, 9, 15, 17])
@pytest.mark.parametrize("groups,rows", [(3, 40), (300, 9), (1, 1)])
def test_group_norm_narrow_groups(io, n, groups, rows, gate):
    """Several rows a workgroup, more groups than a workgroup has places, and one group alone."""
    for rms, bias, silu in ((False, True, True), (True, False, True), (False, True, False)):
        c = group_inputs(io, 1, rows, n * groups, groups, gate, bias, 331, wide=n % 2 == 0)
        out = group_both(c, groups, gate, silu, rms)
        sync()
        check_group(io, c, groups, gate, silu, rms, None, *out)


@pytest.mark.parametrize("gate", ["none", "after", "before"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,groups", [(1, 7), (2, 5), (3, 5), (4, 5), (5, 5), (7, 3)])
def test_group_norm_narrow_groups_of_many_rows(io, n, groups, gate):
    """More rows than the GPU takes at once; run to run the same bits."""
    L = 9001
    c = group_inputs(io, 2, L, n * groups, groups, gate, True, 332)
    lens = [L, L // 3]
    one, two = (group_both(c, groups, gate, True, False, i32(lens)) for _ in range(2))
    sync()
    assert all(same(a, b) for a, b in zip(outputs(one), outputs(two)))
    check_group(io, c, groups, gate, True, False, lens, *one, rows_depth=256)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 3, 5, 7])
def test_group_norm_narrow_groups_padding_and_bad_values(io, n):
    """Groups whose pieces overlap: padding reaches nothing, and a bad group stays alone."""
    import torch
    B, L, G = 3, 20, 9
    lens = [20, 7, 0]
    for gate in ("none", "after", "before"):
        c = group_inputs(io, B, L, n * G, G, gate, True, 333, wide=False)
        want = outputs(group_both(c, G, gate, True, False, i32(lens)))
        k = {name: None if t is None else t.clone() for name, t in c.items()}
        for name in ("x", "dy") + (("z",) if gate != "none" else ()):
            for b, m in enumerate(lens):
                k[name][b, m:] = float("nan")
        assert all(same(a, b) for a, b in zip(outputs(group_both(k, G, gate, True, False, i32(lens))), want))
        k = dict(c, x=c["x"].clone())
        k["x"][1, 2, 4 * n] = float("nan")
        got = outputs(group_both(k, G, gate, True, False, i32(lens)))
        keep = torch.ones((B, L, n * G), dtype=torch.bool, device=DEV)
        keep[1, 2, 4 * n:5 * n] = False
        for a, b in ((got[0], want[0]), (got[3], want[3])):
            assert same(a[keep], b[keep]) and torch.isnan(a[~keep]).all()
