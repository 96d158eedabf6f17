"""The gated recurrence and the group norm on the GPU against the 64-bit reference
of recurrent_ref.py, element by element within its counted tolerances, and their
edge cases: rows of no and one step, padding that holds NaN and infinities,
strides, odd widths, caches with idle and repeated slots, other streams, graphs,
offsets past 32 bits, and the operators together as a block that trains and
serves."""
import numpy as np
import pytest

import recurrent_ref as R
from block_ref import check, lengths
from test_gpu_block import DEV, Gen, _dt, _near, bits, i32, n64, sync

pytestmark = pytest.mark.gpu

CHUNK = 64


def off(t, offset):
    """A copy that starts inside its allocation, at no multiple of 16 bytes."""
    import torch
    flat = torch.zeros(t.numel() + offset, dtype=t.dtype, device=DEV)
    v = flat[offset:].view(t.shape)
    v.copy_(t)
    return v


# ---- gated recurrence --------------------------------------------------------

def gated_inputs(io, B, L, D, seed, wide=False, carry=True, rate=None):
    g = Gen(seed, io)
    gates = g.normal(B, L, 2 * D)
    ag, xg = (gates[..., :D], gates[..., D:]) if wide else (gates[..., :D].contiguous(), gates[..., D:].contiguous())
    import torch
    A = torch.rand(D, generator=g.g) * 6 - 5 if rate is None else torch.full((D,), float(rate))
    return dict(x=g.normal(B, L, D), ag=ag, xg=xg, A=A.to(DEV), h0=g.normal(B, D, io="f32") if carry else None,
                dy=g.normal(B, L, D), dl=g.normal(B, D, io="f32") if carry else None)


def gated_both(c, valid_len=None, **kw):
    """Forward and backward: y, h_last, chunk_states and the gradients."""
    import selective_state_space_scan_amd as ssm
    y, last, st = ssm.gated_recurrence_fwd(c["x"], c["ag"], c["xg"], c["A"], valid_len, h0=c["h0"],
                                           return_chunk_states=True)
    g = ssm.gated_recurrence_bwd(c["x"], c["ag"], c["xg"], c["A"], valid_len, c["dy"], st, h0=c["h0"], dh_last=c["dl"], **kw)
    return y, last, st, g


def check_gated(io, c, lens, y, last, st, g):
    a = (n64(c["x"]), n64(c["ag"]), n64(c["xg"]), n64(c["A"]), lens)
    ref, tol = R.gated_fwd(*a, n64(c["h0"]), io)
    for name, got, r, t in zip(("y", "h_last", "chunk_states"), (y, last, st), ref, tol):
        if got is not None:
            check(name, n64(got), r, t)
    if g is not None:
        ref, tol = R.gated_bwd(*a, n64(c["dy"]), n64(c["h0"]), n64(c["dl"]), io)
        for k in ("dx", "da_gate", "dx_gate", "dA_log") + (("dh0",) if c["h0"] is not None else ()):
            check(k, n64(g[k]), ref[k], tol[k])
        assert (g["dh0"] is None) == (c["h0"] is None)
    B, L, _ = c["x"].shape
    for b, n in enumerate(lengths(lens, B, L)):
        for t in [y] + ([] if g is None else [g["dx"], g["da_gate"], g["dx_gate"]]):
            assert not bits(t)[b, n:].any()   # +0


GATED = [
    # io, B, L, D, lens
    ("f32", 2, 37, 64, None),
    ("bf16", 3, 70, 72, [70, 33, 0]),
    ("bf16", 4, 9, 13, [1, 2, 3, 9]),
    ("f32", 3, 5, 7, [0, 1, 5]),
    ("f32", 1, 1, 1, None),
    ("bf16", 2, 1, 8, [1, 0]),
    ("bf16", 1, 133, 1030, None),
    ("f32", 2, 260, 33, [-4, 999]),
    ("bf16", 2, 600, 24, [513, 600]),
    ("f32", 5, 64, 130, [64, 63, 32, 31, 33]),
    ("bf16", 2, 129, 129, [128, 65]),
    ("f32", 2, 300, 65, [257, 192]),
    ("bf16", 1, 1025, 2, None),
    ("bf16", 2, 513, 1, [512, 511]),
    ("f32", 1, 2100, 201, [2049]),
]


@pytest.mark.parametrize("carry,wide", [(True, True), (False, False)])
@pytest.mark.parametrize("io,B,L,D,lens", GATED)
def test_gated(io, B, L, D, lens, carry, wide):
    import torch
    c = gated_inputs(io, B, L, D, 111, wide, carry)
    kw = {}
    if wide:
        buf = torch.full((B, L, 3 * D), 7.0, dtype=_dt(io), device=DEV)
        kw = dict(da_gate=buf[..., :D], dx_gate=buf[..., D:2 * D])
    y, last, st, g = gated_both(c, i32(lens), **kw)
    sync()
    check_gated(io, c, lens, y, last, st, g)
    if wide:
        assert g["da_gate"].data_ptr() == buf.data_ptr() and (buf[..., 2 * D:] == 7).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,lens", [
    (5, 3500, 201, [3500, 3487, 12, 0, 1777]),      # rows of every kind of length, an odd width
    (1, 9000, 130, None),                           # one long row
    (2, 4096, 64, [4096, 2048]),                    # whole tiles, a narrow width
    (70, 200, 66, None),                            # many short rows
])
def test_gated_large(io, B, L, D, lens):
    """Work enough for every way that rows are cut up, run to run the same bits."""
    c = gated_inputs(io, B, L, D, 118)
    one, two = gated_both(c, i32(lens)), gated_both(c, i32(lens))
    sync()
    check_gated(io, c, lens, *one)
    for a, b in zip((*one[:3], *one[3].values()), (*two[:3], *two[3].values())):
        assert np.array_equal(bits(a), bits(b))


@pytest.mark.parametrize("io,B,L,D,lens", [
    ("bf16", 8, 8197, 130, [8197, 8197, 0, 1, 256, 4096, 4097, 8190]),  # tiles of 16 waves, two channels a lane
    ("f32", 8, 8197, 130, None),
    ("bf16", 17, 8200, 63, [8200 - 511 * b for b in range(17)]),        # the same, one channel
    ("f32", 8, 4100, 129, [4100, 0, 0, 0, 0, 0, 0, 4099]),              # of eight, rows of padding alone between
    ("bf16", 8, 4100, 130, None),
    ("bf16", 1, 20000, 18, None),                                       # more than nine spans
    ("bf16", 1, 2101, 16385, [1500]),                                   # backward tiles dealt in pairs, an odd number
    ("f32", 2, 2090, 8200, [2090, 33]),
    *[("bf16", 530, L, 66, None) for L in (3, 17, 100)],                # whole rows, two channels a lane
    ("f32", 530, 40, 66, [b % 43 - 1 for b in range(530)]),
    ("bf16", 130, 250, 66, [b * 2 for b in range(130)]),
    *[("f32", 513, L, 3, None) for L in (16, 31, 64, 120)],             # one
    *[(io, 2, L, 19, None) for L in (32, 33, 65, 129, 257, 511, 512) for io in ("f32", "bf16")],  # sixteen channels
    *[(io, 2, L, 35, [L, 530]) for L in (513, 1000, 1024) for io in ("f32", "bf16")],   # sixteen steps a lane
])
def test_gated_every_cut(io, B, L, D, lens):
    """Every way that rows are cut up, in full and with rows that end early, run to run the same bits."""
    c = gated_inputs(io, B, L, D, 161, carry=B != 8)
    one, two = gated_both(c, i32(lens)), gated_both(c, i32(lens))
    sync()
    check_gated(io, c, lens, *one)
    for a, b in zip((*one[:3], *one[3].values()), (*two[:3], *two[3].values())):
        assert a is b is None or np.array_equal(bits(a), bits(b))


@pytest.mark.parametrize("B,L,D", [(600, 20, 129), (5, 600, 257), (9, 4100, 129), (2, 100, 17), (520, 100, 67)])
def test_gated_state_in_place(B, L, D):
    """h_last in h0's place: read before it is written, also where lanes share a channel."""
    import selective_state_space_scan_amd as ssm
    c = gated_inputs("bf16", B, L, D, 162)
    y, last = ssm.gated_recurrence_fwd(c["x"], c["ag"], c["xg"], c["A"], h0=c["h0"])[:2]
    h = c["h0"].clone()
    y2, last2 = ssm.gated_recurrence_fwd(c["x"], c["ag"], c["xg"], c["A"], h0=h, h_last=h)[:2]
    assert last2.data_ptr() == h.data_ptr()
    assert np.array_equal(bits(y), bits(y2)) and np.array_equal(bits(last), bits(h))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_lengths_around_every_edge(io):
    """A row for every length around waves, chunks and tiles."""
    lens = sorted({n + d for n in (0, 8, 16, 32, 64, 128, 192, 256, 384, 512, 640) for d in (-1, 0, 1) if n + d >= 0})
    c = gated_inputs(io, len(lens), 641, 5, 119)
    y, last, st, g = gated_both(c, i32(lens))
    sync()
    check_gated(io, c, lens, y, last, st, g)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [-30.0, -12.0, 3.0, 20.0])
def test_gated_decays_of_every_size(io, rate):
    """Channels that hardly forget (1 - a^2 far below a's step) and ones that forget at once (a underflows)."""
    c = gated_inputs(io, 2, 150, 70, 120, rate=rate)
    y, last, st, g = gated_both(c, None)
    sync()
    check_gated(io, c, None, y, last, st, g)


def test_gated_decays_at_their_ends():
    """exp(A_log) of 0 keeps the state and lets nothing in, an infinite one passes the gated input alone; gradients
    through the decay are their limit 0; open and closed gates."""
    import torch
    B, L, D = 1, 80, 6
    c = gated_inputs("f32", B, L, D, 121)
    c["A"] = torch.tensor([-float("inf"), -200.0, 100.0, float("inf"), 0.0, 0.0], device=DEV)
    c["ag"][..., 4], c["xg"][..., 4] = 200.0, -200.0   # forgets by e^-1 a step, nothing comes in
    c["ag"][..., 5], c["xg"][..., 5] = -200.0, 200.0   # keeps everything, and so lets nothing in
    y, last, st, g = gated_both(c, None)
    sync()
    y, h0, x, xg = n64(y)[0], n64(c["h0"])[0], n64(c["x"])[0], n64(c["xg"])[0]
    for d in (0, 1, 5):
        assert (y[:, d] == h0[d]).all()
    for d in (2, 3):
        want = x[:, d] / (1 + np.exp(-xg[:, d]))
        check("y", y[:, d], want, 16 * R.U * np.abs(want))
    want = h0[4] * np.exp(-np.arange(1.0, L + 1))
    check("y", y[:, 4], want, 16 * L * R.U * np.abs(want) + 1e-37)
    for k in ("dx", "da_gate", "dx_gate", "dA_log", "dh0"):
        assert torch.isfinite(g[k]).all(), k
    assert (g["dA_log"][[0, 1, 2, 3, 5]] == 0).all() and (g["da_gate"][..., :4] == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_padding_reaches_nothing(io):
    """NaN, infinities and the type's lowest value past a row's end change no bit."""
    import torch
    B, L, D = 5, 300, 40
    lens = [300, 140, 1, 0, 256]
    c = gated_inputs(io, B, L, D, 113)
    vl = i32(lens)

    def all_bits(c):
        y, last, st, g = gated_both(c, vl)
        return [bits(t) for t in (y, last, st, *g.values())]

    want = all_bits(c)
    for bad in (float("nan"), float("inf"), torch.finfo(_dt(io)).min):
        k = {n: t.clone() for n, t in c.items()}
        for b, n in enumerate(lens):
            for name in ("x", "ag", "xg", "dy"):
                k[name][b, n:] = bad
        for a, b in zip(all_bits(k), want):
            assert np.array_equal(a, b)


def test_gated_bad_values_stay_in_their_channel_and_row():
    import torch
    B, L, D = 2, 400, 131
    c = gated_inputs("f32", B, L, D, 114)
    good = gated_both(c)
    for name in ("x", "ag", "xg", "dy"):
        k = {n: t.clone() for n, t in c.items()}
        k[name][0, 200, 7], k[name][0, 200, 130] = float("nan"), float("nan")
        bad = gated_both(k)
        ok = [d for d in range(D) if d not in (7, 130)]
        for a, b in zip((*bad[:3], bad[3]["dx"], bad[3]["da_gate"], bad[3]["dx_gate"], bad[3]["dh0"]),
                        (*good[:3], good[3]["dx"], good[3]["da_gate"], good[3]["dx_gate"], good[3]["dh0"])):
            assert torch.equal(a[..., ok], b[..., ok]) and torch.equal(a[1], b[1])
        assert torch.equal(bad[3]["dA_log"][ok], good[3]["dA_log"][ok])
        if name != "dy":   # the state forgets a NaN never, and knows nothing of it before it comes
            assert torch.isnan(bad[0][0, 200:, 7]).all() and torch.equal(bad[0][0, :200], good[0][0, :200])
    # an infinite input: the state is infinite from there on
    k = {n: t.clone() for n, t in c.items()}
    k["x"][0, 200, 7] = float("inf")
    y = gated_both(k)[0]
    assert torch.isposinf(y[0, 200:, 7]).all() and torch.equal(y[0, :200], good[0][0, :200])


@pytest.mark.parametrize("offset", [1, 3])
def test_gated_unaligned_views(offset):
    import torch
    c = gated_inputs("bf16", 2, 200, 24, 116)
    o = {k: off(t, offset) for k, t in c.items()}
    for a, b in zip(gated_both(c)[:3], gated_both(o)[:3]):
        assert torch.equal(a, b)
    a, b = gated_both(c)[3], gated_both(o, dx=off(c["x"], offset))[3]
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_gated_time_major_and_repeated_inputs():
    """Tensors as [L, B, D] buffers seen as [B, L, D]; inputs with stride 0."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D = 3, 150, 24
    c = gated_inputs("bf16", B, L, D, 115)
    tm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    want = gated_both(c)
    m = {k: tm(t) if t.dim() == 3 else t for k, t in c.items()}
    got = gated_both(m, dx=tm(torch.zeros_like(c["x"])))
    y, last = ssm.gated_recurrence_fwd(m["x"], m["ag"], m["xg"], m["A"], h0=m["h0"], y=tm(torch.zeros_like(c["x"])))
    assert y.stride() == m["x"].stride() and torch.equal(y, want[0]) and torch.equal(last, want[1])
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    assert all(torch.equal(got[3][k], want[3][k]) for k in want[3])
    r = dict(c, x=c["x"][:1].expand(B, L, D), ag=c["ag"][:, :1].expand(B, L, D), dy=c["dy"][:1, :1].expand(B, L, D))
    s = {k: t.contiguous() for k, t in r.items()}
    a, b = gated_both(r), gated_both(s)
    assert all(torch.equal(x, y) for x, y in zip((*a[:3], *a[3].values()), (*b[:3], *b[3].values())))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_in_pieces(io):
    """A sequence cut anywhere and carried on, the state updated in place, is the whole sequence within its counted
    error; the state of a row that ends before the cut passes through bit by bit."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D = 3, 700, 72
    c = gated_inputs(io, B, L, D, 117)
    lens = [700, 90, 350]
    (ry, rl, _), (ty, tl, _) = R.gated_fwd(n64(c["x"]), n64(c["ag"]), n64(c["xg"]), n64(c["A"]), lens, n64(c["h0"]), io)
    for cut in (1, 64, 351, 699):
        h = c["h0"].clone()
        ys = []
        for part in (slice(0, cut), slice(cut, L)):
            vl = i32([min(max(n - part.start, 0), part.stop - part.start) for n in lens])
            before = h.clone()
            y, back = ssm.gated_recurrence_fwd(c["x"][:, part], c["ag"][:, part], c["xg"][:, part], c["A"], vl, h0=h, h_last=h)
            assert back is h
            for b in range(B):
                if int(vl[b]) == 0:
                    assert torch.equal(h[b], before[b])
            ys.append(y)
        sync()
        check("y", n64(torch.cat(ys, 1)), ry, ty)
        check("h_last", n64(h), rl, tl)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_empty(io):
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(127, io)
    A, h0 = g.normal(8, io="f32"), g.normal(3, 8, io="f32")
    x = torch.empty((3, 0, 8), dtype=_dt(io), device=DEV)
    y, last, st = ssm.gated_recurrence_fwd(x, x, x, A, h0=h0, return_chunk_states=True)   # no steps: the state stays
    assert y.shape == x.shape and torch.equal(last, h0) and st.shape == (3, 0, 8)
    assert (ssm.gated_recurrence_fwd(x, x, x, A)[1] == 0).all()
    assert torch.equal(ssm.gated_recurrence_fwd(x, x, x, A, h0=h0, h_last=h0)[1], last)
    r = ssm.gated_recurrence_bwd(x, x, x, A, None, x, st, h0=h0, dh_last=h0)
    assert torch.equal(r["dh0"], h0) and (r["dA_log"] == 0).all()
    x = torch.empty((0, 5, 8), dtype=_dt(io), device=DEV)
    y, last = ssm.gated_recurrence_fwd(x, x, x, A)
    assert y.numel() == 0 and last.shape == (0, 8)
    assert (ssm.gated_recurrence_bwd(x, x, x, A, None, x, None)["dA_log"] == 0).all()
    x = torch.empty((2, 5, 0), dtype=_dt(io), device=DEV)
    assert ssm.gated_recurrence_fwd(x, x, x, A[:0])[0].numel() == 0
    assert ssm.gated_recurrence_bwd(x, x, x, A[:0], None, x, None)["dA_log"].shape == (0,)
    x = g.normal(2, 70, 8)   # only rows of no steps
    y, last, st = ssm.gated_recurrence_fwd(x, x, x, A, i32([0, -3]), h0=h0[:2], return_chunk_states=True)
    assert not bits(y).any() and torch.equal(last, h0[:2]) and all(torch.equal(st[:, k], h0[:2]) for k in (0, 1))
    r = ssm.gated_recurrence_bwd(x, x, x, A, i32([0, -3]), x, st, h0=h0[:2], dh_last=h0[1:])
    assert torch.equal(r["dh0"], h0[1:]) and (r["dA_log"] == 0).all() and not bits(r["dx"]).any()


# ---- single tokens -----------------------------------------------------------

@pytest.mark.parametrize("io,B,D,slots", [
    ("f32", 1, 64, None), ("bf16", 3, 72, None), ("bf16", 5, 13, [6, 0, -1, 2, 5]), ("f32", 4, 7, [7, 3, 8, 100]),
    ("bf16", 6, 2057, [3, 1, 3, 0, 1, -7]), ("f32", 1, 1, [0]), ("f32", 7, 1030, [1, 2, 3, 4, 5, 6, 7])])
def test_gated_step(io, B, D, slots):
    import torch
    import selective_state_space_scan_amd as ssm
    c = gated_inputs(io, B, 1, D, 122, wide=True)
    n = B if slots is None else 8
    h = Gen(123, "f32").normal(n, D)
    x, ag, xg = (c[k][:, 0] for k in ("x", "ag", "xg"))
    new = torch.full_like(h, 9.0)
    wide = torch.full((B, 2 * D), 5.0, dtype=_dt(io), device=DEV)
    y = ssm.gated_recurrence_step(x, ag, xg, c["A"], h, slots=i32(slots), h_last=new, y=wide[:, :D])
    inplace = h.clone()
    y2 = ssm.gated_recurrence_step(x, ag, xg, c["A"], inplace, slots=i32(slots))
    sync()
    live, seen = [], set()
    for i in range(B):
        s = i if slots is None else slots[i]
        if 0 <= s < n and s not in seen:
            live.append((i, s))
            seen.add(s)
    rows, at = [i for i, _ in live], [s for _, s in live]
    (ry, rl, _), (ty, tl, _) = R.gated_fwd(n64(c["x"])[rows], n64(c["ag"])[rows], n64(c["xg"])[rows], n64(c["A"]), None,
                                          n64(h)[at], io)
    check("y", n64(y)[rows], ry[:, 0], ty[:, 0])
    check("h_last", n64(new)[at], rl, tl)
    idle = [i for i in range(B) if i not in rows]
    rest = [s for s in range(n) if s not in seen]
    assert not bits(y)[idle].any() and (n64(new)[rest] == 9).all() and (wide[:, D:] == 5).all()
    assert torch.equal(y, y2) and torch.equal(inplace[at], new[at]) and torch.equal(inplace[rest], h[rest])


def test_gated_step_idle_rows_and_repeated_slots():
    """What an idle row's inputs hold reaches no output, an empty cache leaves every row idle, and of rows that name
    one slot the first takes the step, among more rows than a wave has lanes."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(124, "f32")
    B, D = 901, 330
    x, ag, xg, A, h = g.normal(B, D), g.normal(B, D), g.normal(B, D), g.normal(D), g.normal(300, D)
    order = torch.cat([torch.randperm(300, generator=g.g) for _ in range(3)] + [torch.tensor([7])]).to(DEV, torch.int32)
    h1, h2 = h.clone(), h.clone()
    y = ssm.gated_recurrence_step(x, ag, xg, A, h1, slots=order)
    y2 = ssm.gated_recurrence_step(x[:300], ag[:300], xg[:300], A, h2, slots=order[:300])
    assert torch.equal(h1, h2) and torch.equal(y[:300], y2) and (y[300:] == 0).all()
    x[1] = float("nan")
    h1 = h.clone()
    y = ssm.gated_recurrence_step(x[:3], ag[:3], xg[:3], A, h1, slots=i32([2, -1, 0]))
    assert torch.isfinite(y).all() and torch.isfinite(h1).all()
    assert (ssm.gated_recurrence_step(x[:3], ag[:3], xg[:3], A, h[:0], slots=i32([2, -1, 0])) == 0).all()
    assert ssm.gated_recurrence_step(x[:0], ag[:0], xg[:0], A, h, slots=i32([])).shape == (0, D)
    B = 65535
    x = g.normal(B + 1, 8)
    h = g.normal(B + 1, 8)
    h1 = h[:B].clone()
    y = ssm.gated_recurrence_step(x[:B], x[:B], x[:B], A[:8], h1)
    assert torch.equal(y, h1)
    half = ssm.gated_recurrence_step(x[B // 2:B], x[B // 2:B], x[B // 2:B], A[:8], h[B // 2:B].clone())
    assert torch.equal(y[B // 2:], half)
    with pytest.raises(ssm.SsmScanError) as e:
        ssm.gated_recurrence_step(x, x, x, A[:8], h)
    assert e.value.code == ssm.SSM_ERR_UNSUPPORTED


# ---- group norm --------------------------------------------------------------

GROUP = [
    # io, B, L, D, groups, lens
    ("f32", 2, 9, 64, 4, None),
    ("bf16", 3, 20, 72, 3, [20, 7, 0]),
    ("bf16", 4, 3, 13, 13, [1, 2, 3, 0]),      # groups of one channel
    ("f32", 1, 1, 1, 1, None),
    ("f32", 3, 5, 35, 7, [0, 1, 5]),
    ("bf16", 2, 6, 1000, 8, [6, 3]),
    ("f32", 1, 11, 600, 12, None),
    ("bf16", 1, 4, 2050, 1, None),
    ("bf16", 2, 3, 130 * 16, 130, None),       # more groups than a workgroup has places
    ("f32", 1, 3, 33 * 40, 33, None),
    ("bf16", 1, 5, 96, 2, [-3]),
]
GATES = [("none", True), ("none", False), ("after", True), ("after", False), ("before", True), ("before", False)]


def group_inputs(io, B, L, D, groups, gate, bias, seed, wide=True, shift=0.3):
    g = Gen(seed, io)
    z = None
    if gate != "none":
        z = g.normal(B, L, 2 * D)[..., D:] if wide else g.normal(B, L, D)
    return dict(x=g.normal(B, L, 3 * D, scale=2.0, shift=shift)[..., D:2 * D] if wide
                else g.normal(B, L, D, scale=2.0, shift=shift), z=z, w=g.normal(D, io="f32", shift=1.0),
                b=g.normal(D, io="f32") if bias else None, dy=g.normal(B, L, D))


def group_both(c, groups, gate, silu, rms, valid_len=None, **kw):
    import selective_state_space_scan_amd as ssm
    f = dict(z=c["z"], silu=silu, gate_first=gate == "before")
    y, m, r = ssm.group_norm_fwd(c["x"], groups, c["w"], c["b"], valid_len, **f, rms=rms, return_stats=True)
    g = ssm.group_norm_bwd(c["dy"], c["x"], groups, c["w"], c["b"], m, r, valid_len, **f, **kw)
    return y, m, r, g


def check_group(io, c, groups, gate, silu, rms, lens, y, m, r, g, rows_depth=128):
    B, L, D = c["x"].shape
    rows = np.concatenate([np.arange(n) + b * L for b, n in enumerate(lengths(lens, B, L))]).astype(int)
    pad = np.setdiff1d(np.arange(B * L), rows)
    two = lambda t: None if t is None else n64(t).reshape(B * L, -1)  # noqa: E731
    pick = lambda t: None if t is None else two(t)[rows]  # noqa: E731
    f = dict(z=pick(c["z"]), silu=silu, gate_first=gate == "before", io=io)
    ref, tol = R.group_fwd(pick(c["x"]), groups, n64(c["w"]), n64(c["b"]), rms=rms, **f)
    check("y", pick(y), ref[0], tol[0])
    check("rstd", pick(r), ref[2], tol[2])
    assert (m is None) == rms
    if not rms:
        check("mean", pick(m), ref[1], tol[1])
    gref, gtol = R.group_bwd(pick(c["dy"]), pick(c["x"]), groups, n64(c["w"]), n64(c["b"]), pick(m), pick(r),
                             rows_depth=rows_depth, **f)
    check("dx", pick(g["dx"]), gref["dx"], gtol["dx"])
    if gate != "none":
        check("dz", pick(g["dz"]), gref["dz"], gtol["dz"])
    check("dweight", n64(g["dweight"]), gref["dweight"], gtol["dweight"])
    if c["b"] is not None:
        check("dbias", n64(g["dbias"]), gref["dbias"], gtol["dbias"])
    assert (g["dz"] is None) == (gate == "none") and (g["dbias"] is None) == (c["b"] is None)
    for t in (y, r, g["dx"], g["dz"]) + (() if rms else (m,)):
        assert t is None or not bits(t).reshape(B * L, -1)[pad].any()   # +0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gate,silu", GATES)
@pytest.mark.parametrize("io,B,L,D,groups,lens", GROUP)
def test_group_norm(io, B, L, D, groups, lens, gate, silu, rms):
    import torch
    c = group_inputs(io, B, L, D, groups, gate, silu, 131)
    buf = torch.full((B, L, 2 * D), 7.0, dtype=_dt(io), device=DEV)
    out = group_both(c, groups, gate, silu, rms, i32(lens), dx=buf[..., :D])
    sync()
    check_group(io, c, groups, gate, silu, rms, lens, *out)
    assert (buf[..., D:] == 7).all()


@pytest.mark.parametrize("gate", ["none", "after", "before"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,groups,rows", [(8, 3, 40), (16, 40, 9), (40, 12, 30), (64, 16, 37), (100, 5, 21),
                                           (200, 3, 20), (256, 2, 9), (500, 2, 9), (512, 4, 5), (1030, 2, 7),
                                           (2048, 2, 5), (2049, 1, 5), (5000, 2, 3), (8192, 1, 3)])
def test_group_norm_every_width(io, n, groups, rows, gate):
    """Every number of lanes that a group takes, full and not."""
    for rms, bias in ((False, True), (True, False)):
        c = group_inputs(io, 1, rows, n * groups, groups, gate, bias, 132, wide=n % 2 == 0)
        out = group_both(c, groups, gate, True, rms)
        sync()
        check_group(io, c, groups, gate, True, rms, None, *out)


@pytest.mark.parametrize("gate", ["none", "after", "before"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,groups,L", [(8, 5, 9001), (24, 7, 4001), (64, 3, 3001), (130, 2, 2501), (300, 2, 2001),
                                        (1000, 1, 1501)])
def test_group_norm_many_rows(io, n, groups, L, gate):
    """More rows than the GPU takes at once, so a workgroup walks several; run to run the same bits.  Rows behind one
    another in a weight's sum: a lane's, 16 of the second pass's lanes, and the joins."""
    c = group_inputs(io, 2, L, n * groups, groups, gate, True, 133)
    lens = [L, L // 3]
    one, two = (group_both(c, groups, gate, True, False, i32(lens)) for _ in range(2))
    sync()
    check_group(io, c, groups, gate, True, False, lens, *one, rows_depth=256)
    for a, b in zip((*one[:3], *one[3].values()), (*two[:3], *two[3].values())):
        assert (a is None and b is None) or np.array_equal(bits(a), bits(b))


def test_group_norm_is_the_layer_norm_with_one_group():
    """The framework's own layer norm, group by group."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(134, "f32")
    x, w, b = g.normal(50, 96, scale=2.0, shift=0.3), g.normal(96), g.normal(96)
    for rms in (False, True):
        y, m, r = ssm.group_norm_fwd(x, 3, w, b, silu=False, rms=rms, return_stats=True)
        for k in range(3):
            s = slice(32 * k, 32 * k + 32)
            ly, _, lm, lr = ssm.layer_norm_fwd(x[:, s].contiguous(), w[s].contiguous(), b[s].contiguous(), rms=rms,
                                               return_stats=True)
            assert torch.allclose(y[:, s], ly, rtol=1e-6, atol=1e-6) and torch.allclose(r[:, k], lr, rtol=1e-6)
            if not rms:
                assert torch.allclose(m[:, k], lm, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_group_norm_padding_reaches_nothing(io):
    """NaN, infinities and the type's lowest value past a row's end, and weights that are not finite: padded rows stay
    +0, and valid ones are as they were."""
    import torch
    B, L, D, G = 4, 15, 40, 5
    lens = [15, 8, 1, 0]
    vl = i32(lens)
    for gate in ("none", "after", "before"):
        c = group_inputs(io, B, L, D, G, gate, True, 135, wide=False)
        flat = lambda o: [bits(t) for t in (*o[:3], *o[3].values()) if t is not None]  # noqa: E731
        want = flat(group_both(c, G, gate, True, False, vl))
        for bad in (float("nan"), float("inf"), torch.finfo(_dt(io)).min):
            k = {n: None if t is None else t.clone() for n, t in c.items()}
            for b, n in enumerate(lens):
                for name in ("x", "dy") + (("z",) if gate != "none" else ()):
                    k[name][b, n:] = bad
            for a, e in zip(flat(group_both(k, G, gate, True, False, vl)), want):
                assert np.array_equal(a, e)
        k = dict(c, w=c["w"].clone(), b=c["b"].clone())
        k["w"][3], k["w"][12], k["b"][30] = float("inf"), float("nan"), float("-inf")
        y, m, r, g = group_both(k, G, gate, True, False, vl)
        for t in (y, m, r, g["dx"], g["dz"]):
            for b, n in enumerate(lens):
                assert t is None or not bits(t)[b, n:].any()
        y0, _, _, g0 = group_both(c, G, gate, True, False, vl)
        ok = list(range(16, 24)) + list(range(32, 40))   # the groups with finite weights
        assert torch.equal(y[..., ok], y0[..., ok]) and torch.equal(g["dx"][..., ok], g0["dx"][..., ok])
        assert torch.equal(g["dweight"][ok], g0["dweight"][ok]) and torch.equal(g["dbias"][ok], g0["dbias"][ok])


def test_group_norm_bad_groups_stay_alone():
    import torch
    B, L, D, G = 2, 5, 60, 6
    for gate in ("none", "after", "before"):
        c = group_inputs("f32", B, L, D, G, gate, True, 136, wide=False)
        want = group_both(c, G, gate, True, False)
        k = dict(c, x=c["x"].clone())
        k["x"][1, 2, 23] = float("nan")
        k["x"][0, 1, 59] = float("inf")
        got = group_both(k, G, gate, True, False)
        keep = torch.ones((B, L, D), dtype=torch.bool, device=DEV)
        keep[1, 2, 20:30] = False
        keep[0, 1, 50:60] = False
        for a, b in ((got[0], want[0]), (got[3]["dx"], want[3]["dx"])):
            assert torch.equal(a[keep], b[keep]) and torch.isnan(a[1, 2, 20:30]).all()


@pytest.mark.parametrize("n", [7, 40, 700, 5001])
def test_group_norm_far_from_zero_and_constant(n):
    """Groups whose mean is far from zero, and constant ones, whose variance is what rounding leaves of zero (beside
    eps, so their rstd is only positive and finite)."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(137, "f32")
    x = g.normal(6, 2 * n)
    x[0] += 1e4
    x[1], x[2], x[3] = 3e4, 0.0, -7.7e5
    w, b = g.normal(2 * n), g.normal(2 * n)
    y, m, r = ssm.group_norm_fwd(x, 2, w, b, silu=False, return_stats=True)
    sync()
    ref, tol = R.group_fwd(n64(x), 2, n64(w), n64(b), silu=False)
    check("y", n64(y), ref[0], tol[0])
    check("mean", n64(m), ref[1], tol[1])
    spread = [0, 4, 5]
    check("rstd", n64(r)[spread], ref[2][spread], tol[2][spread])
    assert torch.isfinite(r).all() and (r > 0).all()
    d = ssm.group_norm_bwd(x, x, 2, w, b, m, r, silu=False)
    ref, tol = R.group_bwd(n64(x), n64(x), 2, n64(w), n64(b), n64(m), n64(r), silu=False)
    check("dx", n64(d["dx"]), ref["dx"], tol["dx"])


def test_group_norm_two_and_three_dimensions_and_strides():
    """[rows, dim] and [batch, L, dim] agree; time-major, repeated and unaligned views give the same bits."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D, G = 3, 14, 48, 4
    c = group_inputs("bf16", B, L, D, G, "after", True, 138, wide=False)
    want = group_both(c, G, "after", True, False)
    flat2 = {k: t.reshape(B * L, D) if t is not None and t.dim() == 3 else t for k, t in c.items()}
    tm = {k: t.transpose(0, 1).contiguous().transpose(0, 1) if t.dim() == 3 else t for k, t in c.items()}
    for k in (flat2, tm, {k: off(t, 3) for k, t in c.items()}):
        got = group_both(k, G, "after", True, False)
        for a, b in zip((*got[:3], *got[3].values()), (*want[:3], *want[3].values())):
            assert torch.equal(a.reshape(b.shape), b)
    y = torch.zeros((L, B, D), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    got = ssm.group_norm_fwd(tm["x"], G, c["w"], c["b"], z=tm["z"], y=y)
    assert got is y and torch.equal(got, want[0])
    r = dict(c, x=c["x"][:1].expand(B, L, D), z=c["z"][:, :1].expand(B, L, D), dy=c["dy"][:1, :1].expand(B, L, D))
    a, b = group_both(r, G, "after", True, False), group_both({k: t.contiguous() for k, t in r.items()}, G, "after", True, False)
    assert all(torch.equal(x, y) for x, y in zip((*a[:3], *a[3].values()), (*b[:3], *b[3].values())))


def test_group_norm_empty():
    import torch
    import selective_state_space_scan_amd as ssm
    w = torch.ones(8, device=DEV)
    x = torch.empty((3, 0, 8), device=DEV)
    y, m, r = ssm.group_norm_fwd(x, 2, w, return_stats=True)
    assert y.shape == x.shape and m.shape == (3, 0, 2)
    g = ssm.group_norm_bwd(x, x, 2, w, w, m, r)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    x = torch.empty((2, 5, 0), device=DEV)
    y, m, r = ssm.group_norm_fwd(x, 3, w[:0], return_stats=True, eps=0.25)
    assert y.numel() == 0 and (m == 0).all() and (r == 2).all()
    g = ssm.group_norm_bwd(x, x, 3, w[:0], w[:0], m, r)
    assert g["dx"].shape == x.shape and g["dweight"].shape == (0,) and g["dbias"].shape == (0,)
    y, m, r = ssm.group_norm_fwd(x, 3, w[:0], None, i32([2, 0]), return_stats=True, eps=0.25, rms=True)
    assert m is None and (r[0, :2] == 2).all() and not r[0, 2:].any() and not r[1].any()


# ---- streams, graphs, limits ---------------------------------------------------

def _all_ops(seed=141, L=700):
    """One call of every operator: a list of (name, function of a stream, outputs as tensors)."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, D, G = 3, 136, 4
    c = gated_inputs("bf16", B, L, D, seed, wide=True)
    vl = i32([L, 7, L // 2 + 5])
    n = group_inputs("bf16", B, L, D, G, "after", True, seed + 1)
    st = ssm.gated_recurrence_fwd(c["x"], c["ag"], c["xg"], c["A"], vl, h0=c["h0"], return_chunk_states=True)[2]
    _, m, r = ssm.group_norm_fwd(n["x"], G, n["w"], n["b"], vl, z=n["z"], return_stats=True)
    h = Gen(seed + 2, "f32").normal(8, D)
    h_last, sl = torch.zeros_like(h), i32([5, -1, 2])
    sync()

    def flat(r):
        return [t for t in (r.values() if isinstance(r, dict) else r) if t is not None]

    return [
        ("gated_fwd", lambda s=None: flat(ssm.gated_recurrence_fwd(c["x"], c["ag"], c["xg"], c["A"], vl, h0=c["h0"],
                                                                  return_chunk_states=True, stream=s))),
        ("gated_bwd", lambda s=None: flat(ssm.gated_recurrence_bwd(c["x"], c["ag"], c["xg"], c["A"], vl, c["dy"], st,
                                                                  h0=c["h0"], dh_last=c["dl"], stream=s))),
        ("gated_step", lambda s=None: [ssm.gated_recurrence_step(c["x"][:, 0], c["ag"][:, 0], c["xg"][:, 0], c["A"], h,
                                                                slots=sl, h_last=h_last, stream=s), h_last]),
        ("group_fwd", lambda s=None: flat(ssm.group_norm_fwd(n["x"], G, n["w"], n["b"], vl, z=n["z"], return_stats=True,
                                                            stream=s))),
        ("group_bwd", lambda s=None: flat(ssm.group_norm_bwd(n["dy"], n["x"], G, n["w"], n["b"], m, r, vl, z=n["z"],
                                                            stream=s))),
    ]


def test_other_streams():
    """A torch stream, a raw stream handle and the current stream give the same bits."""
    import torch
    ops = _all_ops()
    want = {k: [t.clone() for t in f()] for k, f in ops}
    sync()
    s = torch.cuda.Stream()
    for name, f in ops:
        for how in (s, s.cuda_stream):
            got = f(how)
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[name])), name
        with torch.cuda.stream(s):
            got = f()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[name])), name


def test_two_streams_at_once():
    import torch
    sets = [_all_ops(141), _all_ops(151)]
    want = [{k: [t.clone() for t in f()] for k, f in ops} for ops in sets]
    sync()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [{}, {}]
    for _ in range(5):
        for i in (0, 1):
            for name, f in sets[i]:
                got[i][name] = f(streams[i])
    sync()
    for i in (0, 1):
        for name in want[i]:
            assert all(torch.equal(a, b) for a, b in zip(got[i][name], want[i][name])), (i, name)


@pytest.mark.parametrize("L", [150, 2500])
def test_graph_replays(L):
    """Forward, backward and step captured, replayed on changed inputs with eager work between, equal the eager calls."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, D, G = 2, 136, 4
    c = gated_inputs("bf16", B, L, D, 161, wide=True)
    z, w, b = Gen(162, "bf16").normal(B, L, D), Gen(163, "f32").normal(D), Gen(164, "f32").normal(D)
    vl, sl, h, outs = i32([L, 11]), i32([3, 1]), Gen(165, "f32").normal(4, D), torch.zeros((4, D), device=DEV)

    def run():
        y, last, st, g = gated_both(c, vl)
        n, m, r = ssm.group_norm_fwd(y, G, w, b, vl, z=z, return_stats=True)
        gn = ssm.group_norm_bwd(c["dy"], y, G, w, b, m, r, vl, z=z)
        ys = ssm.gated_recurrence_step(c["x"][:, 0], c["ag"][:, 0], c["xg"][:, 0], c["A"], h, slots=sl, h_last=outs)
        return [y, last, st, *g.values(), n, m, r, *gn.values(), ys, outs]

    run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = run()
    g = torch.Generator().manual_seed(166)
    for k in range(4):
        for t in (c["x"], c["ag"], c["xg"], c["dy"], c["h0"], z, h):
            t.copy_(torch.randn(t.shape, generator=g).to(t))
        vl.copy_(i32([L - 40 * k, 11 * k]))
        sl.copy_(i32([k, (k + 1) % 4 if k != 2 else -1]))
        outs.zero_()
        graph.replay()
        sync()
        got = [t.clone() for t in static]
        outs.zero_()
        want = run()
        sync()
        for i, (a, e) in enumerate(zip(got, want)):
            assert torch.equal(a, e), (k, i)


def test_two_graphs_at_once():
    """Two captured training steps, replayed at once on two streams: each has its own scratch."""
    import torch
    graphs, static, want = [], [], []
    for s in (171, 172):
        c = gated_inputs("bf16", 2, 2500, 136, s)
        n = group_inputs("bf16", 2, 2500, 136, 4, "before", True, s)

        def run():
            y, last, st, g = gated_both(c)
            o = group_both(n, 4, "before", True, False)
            return [y, last, st, *g.values(), *o[:3], *o[3].values()]

        want.append([t.clone() for t in run()])
        sync()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            static.append(run())
        static[-1].append((c, n))   # the graph's inputs live as long as it does
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for ts in static:
            for t in ts[:-1]:
                t.zero_()
        sync()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        sync()
        for got, w in zip(static, want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_given_outputs_and_scratch():
    """Outputs and scratch that the caller owns are the ones written and returned; scratch may hold anything."""
    import torch
    import selective_state_space_scan_amd as ssm
    c = gated_inputs("bf16", 2, 2500, 136, 181)
    y0, l0, st, g0 = gated_both(c)
    for fill in (255, 0, 1):
        ws = torch.full((8 << 20,), fill, dtype=torch.uint8, device=DEV)
        y, last = torch.zeros_like(y0), torch.zeros_like(l0)
        r = ssm.gated_recurrence_fwd(c["x"], c["ag"], c["xg"], c["A"], h0=c["h0"], y=y, h_last=last, workspace=ws)
        assert len(r) == 2 and r[0] is y and r[1] is last and torch.equal(y, y0) and torch.equal(last, l0)
        ws.fill_(fill)
        d = [torch.zeros_like(y0) for _ in range(3)]
        g = ssm.gated_recurrence_bwd(c["x"], c["ag"], c["xg"], c["A"], None, c["dy"], st, h0=c["h0"], dh_last=c["dl"],
                                     dx=d[0], da_gate=d[1], dx_gate=d[2], workspace=ws)
        assert g["dx"] is d[0] and g["da_gate"] is d[1] and g["dx_gate"] is d[2]
        assert all(torch.equal(g[k], g0[k]) for k in g0)
        n = group_inputs("bf16", 2, 300, 136, 4, "after", True, 182, wide=False)
        want = group_both(n, 4, "after", True, False)
        y = torch.zeros_like(want[0])
        assert ssm.group_norm_fwd(n["x"], 4, n["w"], n["b"], z=n["z"], y=y) is y and torch.equal(y, want[0])
        dx, dz = torch.zeros_like(y), torch.zeros_like(y)
        ws.fill_(fill)
        g = ssm.group_norm_bwd(n["dy"], n["x"], 4, n["w"], n["b"], want[1], want[2], z=n["z"], dx=dx, dz=dz, workspace=ws)
        assert g["dx"] is dx and g["dz"] is dz and all(torch.equal(g[k], want[3][k]) for k in g)


def test_offsets_past_32_bits():
    """A cache and sequences of more than 2^31 elements: the last rows are as good as the first."""
    import torch
    import selective_state_space_scan_amd as ssm
    D = 2048
    g = Gen(191, "bf16")
    n = 2**31 // D + 9
    h = torch.zeros((n, D), device=DEV)
    x, ag, xg, A, st = g.normal(2, D), g.normal(2, D), g.normal(2, D), g.normal(D, io="f32"), g.normal(2, D, io="f32")
    h[n - 1], h[0] = st[0], st[1]
    y = ssm.gated_recurrence_step(x, ag, xg, A, h, slots=i32([n - 1, 0]))
    y2 = ssm.gated_recurrence_step(x, ag, xg, A, st)
    assert torch.equal(y, y2) and torch.equal(h[n - 1], st[0]) and torch.equal(h[0], st[1])
    assert not h[1:9].any() and not h[n - 9:n - 1].any()
    del h
    # a sequence of 2^31 elements and a bit, compared at its end with a short run from a kept state: the tail is cut
    # where tiles of any length begin
    L = 2**31 // D + 4096
    x = torch.empty((1, L, D), dtype=torch.bfloat16, device=DEV)
    x.view(torch.int16).random_(0x3f00, 0x3fff)   # 0.5 to 2
    A = torch.zeros(D, device=DEV)
    y, last, st = ssm.gated_recurrence_fwd(x, x, x, A, return_chunk_states=True)
    cut = 2**31 // D
    before = st[:, cut // CHUNK - 1].contiguous()
    yt, lt, stt = ssm.gated_recurrence_fwd(x[:, cut:], x[:, cut:], x[:, cut:], A, h0=before, return_chunk_states=True)
    assert torch.allclose(y[:, cut:].float(), yt.float(), rtol=2.0**-7) and torch.allclose(last, lt, rtol=1e-5)
    assert torch.allclose(st[:, cut // CHUNK:], stt, rtol=1e-5)
    r = ssm.gated_recurrence_bwd(x, x, x, A, None, y, st, dh_last=last)
    rt = ssm.gated_recurrence_bwd(x[:, cut:], x[:, cut:], x[:, cut:], A, None, y[:, cut:], stt, h0=before, dh_last=last)
    scale = lambda t: float(t.float().square().mean().sqrt())  # noqa: E731
    for k in ("dx", "da_gate", "dx_gate"):
        assert float((r[k][:, cut:].float() - rt[k].float()).abs().max()) <= 2.0**-6 * max(
            scale(rt[k]), float(rt[k].float().abs().max())), k
    del r, rt, yt
    w = torch.ones(D, device=DEV)
    yn, m, s = ssm.group_norm_fwd(x, 8, w, z=y, return_stats=True)
    tail = slice(L - 50, L)
    yt, mt, rt = ssm.group_norm_fwd(x[:, tail], 8, w, z=y[:, tail], return_stats=True)
    assert torch.equal(yn[:, tail], yt) and torch.equal(m[:, tail], mt) and torch.equal(s[:, tail], rt)
    g = ssm.group_norm_bwd(y, x, 8, w, None, m, s, z=yn)
    gt = ssm.group_norm_bwd(y[:, tail], x[:, tail], 8, w, None, mt.contiguous(), rt.contiguous(), z=yn[:, tail])
    assert torch.equal(g["dx"][:, tail], gt["dx"]) and torch.equal(g["dz"][:, tail], gt["dz"])


def test_many_rows_and_groups():
    """More rows than a grid's side, and a row of very many groups."""
    import torch
    import selective_state_space_scan_amd as ssm
    rows = (1 << 21) + 77
    x, w = torch.randn((rows, 32), device=DEV), torch.ones(32, device=DEV)
    y, m, r = ssm.group_norm_fwd(x, 2, w, return_stats=True)
    for part in (slice(0, 50), slice(rows - 40, rows)):
        yp, mp, rp = ssm.group_norm_fwd(x[part], 2, w, return_stats=True)
        assert torch.equal(y[part], yp) and torch.equal(m[part], mp) and torch.equal(r[part], rp)
    g = ssm.group_norm_bwd(y, x, 2, w, None, m, r)
    gp = ssm.group_norm_bwd(y[-40:], x[-40:], 2, w, None, m[-40:], r[-40:])
    assert torch.equal(g["dx"][-40:], gp["dx"])
    G = 100003
    x, w = torch.randn((3, G * 2), device=DEV), torch.ones(G * 2, device=DEV)
    y, m, r = ssm.group_norm_fwd(x, G, w, silu=False, return_stats=True)
    two = lambda t: t.view(3 * G, 2)  # noqa: E731
    ref, tol = R.group_fwd(n64(two(x)), 1, np.ones(2), None, silu=False)
    check("y", n64(two(y)), ref[0], tol[0])
    g = ssm.group_norm_bwd(x, x, G, w, None, m, r, silu=False)
    ref, tol = R.group_bwd(n64(two(x)), n64(two(x)), 1, np.ones(2), None, n64(m).reshape(-1, 1), n64(r).reshape(-1, 1), silu=False)
    check("dx", n64(two(g["dx"])), ref["dx"], tol["dx"])
    # the batch's largest: as many short rows
    B = 70000
    c = gated_inputs("f32", B, 2, 3, 192)
    y, last, st, g = gated_both(c)
    half = {k: t[B - 50:].contiguous() if k != "A" else t for k, t in c.items()}
    y2, l2, _, g2 = gated_both(half)
    assert torch.equal(y[B - 50:], y2) and torch.equal(last[B - 50:], l2) and torch.equal(g["dx"][B - 50:], g2["dx"])


def test_outputs_that_do_not_fit_are_torch_s_out_of_memory():
    import torch
    import selective_state_space_scan_amd as ssm
    x, w = torch.ones((1, 1, 1024), dtype=torch.bfloat16, device=DEV), torch.ones(1024, device=DEV)
    big = x.expand(1 << 10, 1 << 20, 1024)   # 2 TiB of output
    for f in (lambda: ssm.gated_recurrence_fwd(big, big, big, w), lambda: ssm.group_norm_fwd(big, 8, w)):
        with pytest.raises(torch.OutOfMemoryError):
            f()
    assert torch.isfinite(ssm.gated_recurrence_fwd(x, x, x, w)[0]).all()


def test_written_tensors_count_as_modified():
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(195, "f32")
    B, L, D = 2, 9, 16
    x, x3, A, h, h2 = g.normal(B, D), g.normal(B, L, D), g.normal(D), g.normal(B, D), g.normal(B, D)
    y, y3, a, b, c = (torch.zeros_like(t) for t in (x, x3, x3, x3, x3))
    ins = [x, x3, A]

    def bumped(f, *outs, kept=()):
        old, still = [t._version for t in outs], [t._version for t in (*ins, *kept)]
        f()
        assert all(t._version > v for t, v in zip(outs, old))
        assert [t._version for t in (*ins, *kept)] == still

    bumped(lambda: ssm.gated_recurrence_step(x, x, x, A, h, y=y), h, y)
    bumped(lambda: ssm.gated_recurrence_step(x, x, x, A, h, h_last=h2), h2, kept=(h,))
    bumped(lambda: ssm.gated_recurrence_fwd(x3, x3, x3, A, h0=h, h_last=h, y=y3), h, y3)
    bumped(lambda: ssm.gated_recurrence_fwd(x3, x3, x3, A, h0=h), kept=(h,))
    bumped(lambda: ssm.gated_recurrence_bwd(x3, x3, x3, A, None, x3, None, dx=a, da_gate=b, dx_gate=c), a, b, c)
    bumped(lambda: ssm.group_norm_fwd(x3, 2, A, y=y3), y3)
    _, m, r = ssm.group_norm_fwd(x3, 2, A, z=x3, return_stats=True)
    bumped(lambda: ssm.group_norm_bwd(x3, x3, 2, A, None, m, r, z=x3, dx=a, dz=b), a, b, kept=(m, r))


def test_refusals():
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(196, "bf16")
    D = 16
    x, A, h, t = g.normal(2, 70, D), g.normal(D, io="f32"), g.normal(2, D, io="f32"), g.normal(2, D)
    st = torch.zeros((2, 2, D), device=DEV)
    fwd, bwd, step, gf, gb = (ssm.gated_recurrence_fwd, ssm.gated_recurrence_bwd, ssm.gated_recurrence_step,
                              ssm.group_norm_fwd, ssm.group_norm_bwd)
    m = torch.zeros((2, 70, 4), device=DEV)
    bad = [
        lambda: fwd(x.half(), x, x, A), lambda: fwd(x[0], x[0], x[0], A), lambda: fwd(x, x.float(), x, A),
        lambda: fwd(x, x, x[:, :8], A), lambda: fwd(x, x, x, A.bfloat16()), lambda: fwd(x, x, x, A[:8]),
        lambda: fwd(x.transpose(1, 2), x, x, A), lambda: fwd(x, x, x, A, torch.zeros(2, device=DEV)),
        lambda: fwd(x, x, x, A, torch.zeros(2, dtype=torch.int32)), lambda: fwd(x, x, x, A, h0=h.bfloat16()),
        lambda: fwd(x, x, x, A, h0=h[:1]), lambda: fwd(x, x, x, A, y=x.float()), lambda: fwd(x, x, x, A, h_last=h.t()),
        lambda: fwd(x, x, x, A, workspace=torch.empty(64, device=DEV)), lambda: bwd(x, x, x, A, None, x.float(), st),
        lambda: bwd(x, x, x, A, None, x, st[:, :1]), lambda: bwd(x, x, x, A, None, x, st, dh_last=h[0]),
        lambda: bwd(x, x, x, A, None, x, st, workspace=torch.empty(4, dtype=torch.uint8, device=DEV)),
        lambda: bwd(x, x, x, A, None, x, st, dx=x[..., :1].expand(2, 70, D)),
        lambda: step(x, x, x, A, h), lambda: step(t, t, t, A, h[:1]), lambda: step(t, t, t, A, h.bfloat16()),
        lambda: step(t, t, t, A, h, slots=torch.zeros(2, dtype=torch.int64, device=DEV)),
        lambda: step(t, t, t, A, h, h_last=h[:1]), lambda: gf(x, 3, A), lambda: gf(x, 0, A), lambda: gf(x, -4, A),
        lambda: gf(x, 4, A[:8]), lambda: gf(x, 4, A, A[:8]), lambda: gf(x, 4, A, z=x[:1]), lambda: gf(x, 4, A, z=x.float()),
        lambda: gf(x, 4, A, gate_first=True), lambda: gf(t, 4, A, None, i32([1, 1])), lambda: gf(A, 4, A),
        lambda: gf(x, 4, A, y=x[..., :8]), lambda: gf(x, "a", A), lambda: gf(x, 2.5, A),
        lambda: gb(x.float(), x, 4, A, None, m, m), lambda: gb(x, x, 4, A, None, m, m[0]),
        lambda: gb(x, x, 2, A, None, m, m), lambda: gb(x, x, 4, A, None, m, None), lambda: gb(x, x, 4, A, None, m, m, dz=x),
        lambda: gb(x, x, 4, A, None, m, m, workspace=torch.empty(4, dtype=torch.uint8, device=DEV)),
    ]
    for k in (1.5, "x", None):
        bad.append(lambda k=k: fwd(k, x, x, A))
        bad.append(lambda k=k: gf(k, 4, A))
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            raise AssertionError(i)
    wide = g.normal(2, 8200)
    for f, code in ((lambda: fwd(x, x, x, A, y=x), ssm.SSM_ERR_ALIAS),
                    (lambda: fwd(x, x, x, A, y=torch.zeros_like(x)[:1, :1].expand(2, 70, D)), ssm.SSM_ERR_INVALID_ARG),
                    (lambda: fwd(x, x, x, A, h0=h, h_last=h, y=h.view(torch.bfloat16).view(2, 2, D)[:, :1].expand(2, 70, D)),
                     ssm.SSM_ERR_INVALID_ARG),
                    (lambda: bwd(x, x, x, A, None, x, None), ssm.SSM_ERR_INVALID_ARG),   # 70 steps need their states
                    (lambda: bwd(x, x, x, A, None, x, st, dx=x), ssm.SSM_ERR_ALIAS),
                    (lambda: step(t, t, t, A, h, y=t), ssm.SSM_ERR_ALIAS),
                    (lambda: gf(x, 4, A, y=x), ssm.SSM_ERR_ALIAS), (lambda: gf(x, 4, A, eps=0.0), ssm.SSM_ERR_INVALID_ARG),
                    (lambda: gf(wide, 1, g.normal(8200, io="f32")), ssm.SSM_ERR_UNSUPPORTED)):
        with pytest.raises(ssm.SsmScanError) as e:
            f()
        assert e.value.code == code


# ---- together ------------------------------------------------------------------

class Block:
    """norm -> in-projection -> short convolution -> gates -> gated recurrence -> gated group norm -> out-projection, the
    block that the operators serve, with its forward, its backward and its step on caches, matrix products in float32."""

    def __init__(self, seed, d_model=32, dim=48, W=4, groups=4):
        g = Gen(seed, "f32")
        self.dims = (d_model, dim, W, groups)
        self.p = dict(nw=g.normal(d_model, scale=0.1, shift=1.0), nb=g.normal(d_model, scale=0.1),
                      win=g.normal(2 * dim, d_model, scale=d_model ** -0.5), cw=g.normal(dim, W, scale=0.5),
                      cb=g.normal(dim, scale=0.1), wg=g.normal(2 * dim, dim, scale=dim ** -0.5),
                      A=g.normal(dim, shift=-1.5), gw=g.normal(dim, scale=0.1, shift=1.0), gb=g.normal(dim, scale=0.1),
                      wo=g.normal(d_model, dim, scale=dim ** -0.5))

    def forward(self, x, residual, valid_len):
        import selective_state_space_scan_amd as ssm
        p, (dm, dim, W, G) = self.p, self.dims
        h, v, m, r = ssm.layer_norm_fwd(x, p["nw"], p["nb"], valid_len, residual=residual, return_stats=True)
        xz = h @ p["win"].t()
        xc, conv = ssm.causal_conv_fwd(xz[..., :dim], p["cw"], p["cb"], valid_len, silu=False)
        gates = xc @ p["wg"].t()
        y, state, cs = ssm.gated_recurrence_fwd(xc, gates[..., :dim], gates[..., dim:], p["A"], valid_len,
                                                return_chunk_states=True)
        n, gm, gr = ssm.group_norm_fwd(y, G, p["gw"], p["gb"], valid_len, z=xz[..., dim:], return_stats=True)
        self.saved = (h, v, m, r, xz, xc, gates, y, cs, n, gm, gr)
        return n @ p["wo"].t(), v, conv, state

    def backward(self, dout, dv, valid_len):
        import torch
        import selective_state_space_scan_amd as ssm
        p, (dm, dim, W, G) = self.p, self.dims
        h, v, m, r, xz, xc, gates, y, cs, n, gm, gr = self.saved
        two = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        g = dict(wo=two(dout).t() @ two(n))
        dxz, dgates = torch.empty_like(xz), torch.empty_like(gates)
        q = ssm.group_norm_bwd(dout @ p["wo"], y, G, p["gw"], p["gb"], gm, gr, valid_len, z=xz[..., dim:], dz=dxz[..., dim:])
        s = ssm.gated_recurrence_bwd(xc, gates[..., :dim], gates[..., dim:], p["A"], valid_len, q["dx"], cs,
                                     da_gate=dgates[..., :dim], dx_gate=dgates[..., dim:])
        c = ssm.causal_conv_bwd(xz[..., :dim], p["cw"], p["cb"], valid_len, s["dx"] + dgates @ p["wg"], silu=False,
                                dx=dxz[..., :dim])
        g.update(gw=q["dweight"], gb=q["dbias"], A=s["dA_log"], wg=two(dgates).t() @ two(xc), cw=c["dweight"],
                 cb=c["dbias"], win=two(dxz).t() @ two(h))
        k = ssm.layer_norm_bwd(dxz @ p["win"], v, p["nw"], m, r, valid_len, dresidual_out=dv)
        g.update(nw=k["dweight"], nb=k["dbias"], x=k["dx"])
        return g

    def step(self, x, residual, conv, state, slots):
        import selective_state_space_scan_amd as ssm
        p, (dm, dim, W, G) = self.p, self.dims
        h, v = ssm.layer_norm_fwd(x, p["nw"], p["nb"], residual=residual)
        xz = h @ p["win"].t()
        xc = ssm.causal_conv_step(xz[:, :dim], conv, p["cw"], p["cb"], silu=False, slots=slots)
        gates = xc @ p["wg"].t()
        y = ssm.gated_recurrence_step(xc, gates[:, :dim], gates[:, dim:], p["A"], state, slots=slots)
        return ssm.group_norm_fwd(y, G, p["gw"], p["gb"], z=xz[:, dim:]) @ p["wo"].t(), v


def _block_in_64_bits(p, dims, x, residual, lens):
    """The same block from elementary torch operations in float64 on the CPU, row by row; (out, v) with zeros past a
    row's end."""
    import torch
    dm, dim, W, G = dims
    outs, vs = [], []
    for b, n in enumerate(lens):
        v = x[b, :n] + residual[b, :n]
        c = v - v.mean(1, keepdim=True)
        h = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["nw"] + p["nb"]
        xz = h @ p["win"].t()
        xs = torch.cat([torch.zeros((W - 1, dim), dtype=v.dtype), xz[:, :dim]])
        u = p["cb"] + sum(xs[k:k + n] * p["cw"][:, k] for k in range(W))
        q = u @ p["wg"].t()
        a = torch.exp(-torch.exp(p["A"]) * torch.sigmoid(q[:, :dim]))
        put = torch.sqrt(1 - a * a) * torch.sigmoid(q[:, dim:]) * u
        state, ys = torch.zeros(dim, dtype=v.dtype), []
        for t in range(n):
            state = a[t] * state + put[t]
            ys.append(state)
        y = torch.stack(ys).view(n, G, dim // G)
        y = y - y.mean(2, keepdim=True)
        y = (y / torch.sqrt((y * y).mean(2, keepdim=True) + 1e-5)).view(n, dim) * p["gw"] + p["gb"]
        y = y * xz[:, dim:] * torch.sigmoid(xz[:, dim:])
        outs.append(torch.cat([y @ p["wo"].t(), torch.zeros((x.shape[1] - n, dm), dtype=v.dtype)]))
        vs.append(torch.cat([v, torch.zeros((x.shape[1] - n, dm), dtype=v.dtype)]))
    return torch.stack(outs), torch.stack(vs)


def test_block_trains():
    """The operators in the order of a block's forward and backward, all gradients against automatic differentiation
    of the block in 64 bits."""
    blk = Block(201)
    g = Gen(202, "f32")
    B, L, dm = 3, 145, 32
    lens = [145, 68, 1]
    x, res, dout, dv = (g.normal(B, L, dm) for _ in range(4))
    for b, n in enumerate(lens):
        dout[b, n:] = 0
        dv[b, n:] = 0
    out, v, _, _ = blk.forward(x, res, i32(lens))
    grads = blk.backward(dout, dv, i32(lens))
    sync()
    p = {k: t.double().cpu().requires_grad_() for k, t in blk.p.items()}
    x64 = x.double().cpu().requires_grad_()
    ro, rv = _block_in_64_bits(p, blk.dims, x64, res.double().cpu(), lens)
    ((ro * dout.double().cpu()).sum() + (rv * dv.double().cpu()).sum()).backward()
    _near("out", out, n64(ro))
    _near("v", v, n64(rv))
    for k in grads:
        _near(k, grads[k], n64((x64 if k == "x" else p[k]).grad))


def test_block_serves():
    """Prompts of different lengths through the sequence operators into slots of the caches, then tokens one by one:
    every token's output equals that of the whole sequence in one go."""
    import torch
    blk = Block(203)
    dm, dim, W, G = blk.dims
    g = Gen(204, "f32")
    B, prompt, new = 4, 130, 6
    lens = [130, 2, 67, 1]
    x, res = g.normal(B, prompt + new, dm), g.normal(B, prompt + new, dm)
    _, _, conv, state = blk.forward(x[:, :prompt].contiguous(), res[:, :prompt].contiguous(), i32(lens))
    slots = [5, 0, 7, 3]
    convs, states = torch.full((9, W - 1, dim), 3.0, device=DEV), torch.full((9, dim), 3.0, device=DEV)
    convs[slots], states[slots] = conv, state
    whole_x = torch.zeros((B, prompt + new, dm), device=DEV)
    whole_r = torch.zeros_like(whole_x)
    for b, n in enumerate(lens):
        for dst, src in ((whole_x, x), (whole_r, res)):
            dst[b, :n], dst[b, n:n + new] = src[b, :n], src[b, prompt:]
    whole, _, conv_end, state_end = blk.forward(whole_x, whole_r, i32([n + new for n in lens]))
    sl = i32(slots + [-1])   # the batch is padded by one row
    for t in range(new):
        xt = torch.cat([x[:, prompt + t], torch.zeros((1, dm), device=DEV)])
        rt = torch.cat([res[:, prompt + t], torch.zeros((1, dm), device=DEV)])
        out, _ = blk.step(xt, rt, convs, states, sl)
        sync()
        _near(f"token {t}", out[:B], n64(torch.stack([whole[b, n + t] for b, n in enumerate(lens)])))
    _near("conv", convs[slots], n64(conv_end))
    _near("state", states[slots], n64(state_end))
    rest = [1, 2, 4, 6, 8]
    assert (convs[rest] == 3).all() and (states[rest] == 3).all()


def test_a_second_backward_beside_a_captured_one():
    """A training step captured into a graph while an eager one of the same inputs lives: the calls record no autograd
    graph, so the two share nothing but their inputs."""
    import torch
    c = gated_inputs("bf16", 2, 300, 64, 211)
    eager = gated_both(c)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = gated_both(c)
    for _ in range(3):
        graph.replay()
        again = gated_both(c)
        sync()
        for a, b, e in zip((*static[:3], *static[3].values()), (*again[:3], *again[3].values()),
                           (*eager[:3], *eager[3].values())):
            assert torch.equal(a, e) and torch.equal(b, e)
