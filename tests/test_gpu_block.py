"""The operators beside the scan on the GPU against the 64-bit reference of
block_ref.py, element by element within its counted tolerances, and their edge
cases: rows of no and one step, padding that holds NaN and infinities, strides,
odd widths, caches with idle and repeated slots, other streams, offsets past
32 bits."""
import numpy as np
import pytest

import block_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _dt(io):
    import torch
    return torch.bfloat16 if io == "bf16" else torch.float32


class Gen:
    """Seeded tensors on the GPU, and their exact values in 64 bits on the CPU."""

    def __init__(self, seed, io):
        import torch
        self.g = torch.Generator().manual_seed(seed)
        self.io = io

    def normal(self, *shape, io=None, scale=1.0, shift=0.0):
        import torch
        t = torch.randn(shape, generator=self.g) * scale + shift
        return t.to(_dt(io or self.io)).to(DEV)


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def bits(t):
    import torch
    return t.detach().contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()


def i32(v):
    import torch
    return None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)


def sync():
    import torch
    torch.cuda.synchronize()


# ---- convolution -------------------------------------------------------------

CONV = [
    # io, B, L, D, W, lens
    ("f32", 2, 37, 64, 4, None),
    ("bf16", 3, 70, 72, 4, [70, 33, 0]),
    ("bf16", 4, 9, 13, 4, [1, 2, 3, 9]),
    ("f32", 3, 5, 7, 3, [0, 1, 5]),
    ("f32", 1, 1, 1, 4, None),
    ("bf16", 2, 1, 8, 2, [1, 0]),
    ("bf16", 1, 133, 1030, 3, None),
    ("f32", 2, 260, 33, 2, [-4, 999]),
    ("bf16", 2, 600, 24, 4, [513, 600]),
    ("f32", 5, 64, 520, 4, [64, 63, 32, 31, 33]),
    ("bf16", 2, 40, 3, 4, [40, 5]),
    ("bf16", 1, 70, 2, 3, None),
    ("f32", 1, 20, 5, 4, None),
    ("bf16", 2, 16, 1, 2, [16, 13]),
]


def conv_inputs(io, B, L, D, W, seed, wide=False, bias=True, carry=True):
    g = Gen(seed, io)
    x = g.normal(B, L, 2 * D)[..., D:] if wide else g.normal(B, L, D)
    return dict(x=x, w=g.normal(D, W, io="f32", scale=0.5), b=g.normal(D, io="f32") if bias else None,
                c0=g.normal(B, W - 1, D) if carry else None, dy=g.normal(B, L, D), dl=g.normal(B, W - 1, D))


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("carry,wide", [(True, True), (False, False)])
@pytest.mark.parametrize("io,B,L,D,W,lens", CONV)
def test_conv_fwd(io, B, L, D, W, lens, carry, wide, silu):
    import selective_state_space_scan_amd as ssm
    c = conv_inputs(io, B, L, D, W, 11, wide, bias=silu, carry=carry)
    y, last = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], i32(lens), silu=silu, conv0=c["c0"])
    sync()
    ry, rl, tol = R.conv_fwd(n64(c["x"]), n64(c["w"]), n64(c["b"]), lens, n64(c["c0"]), silu, io)
    R.check("y", n64(y), ry, tol)
    assert np.array_equal(n64(last), rl)
    for b, n in enumerate(R.lengths(lens, B, L)):
        assert not bits(y)[b, n:].any()   # +0


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("carry,wide", [(True, True), (False, False)])
@pytest.mark.parametrize("io,B,L,D,W,lens", CONV)
def test_conv_bwd(io, B, L, D, W, lens, carry, wide, silu):
    import torch
    import selective_state_space_scan_amd as ssm
    c = conv_inputs(io, B, L, D, W, 12, wide, bias=silu, carry=carry)
    dx = torch.full((B, L, 2 * D), 7.0, dtype=_dt(io), device=DEV) if wide else None
    g = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], i32(lens), c["dy"], silu=silu, conv0=c["c0"],
                            dconv_last=c["dl"] if carry else None, dx=None if dx is None else dx[..., :D])
    sync()
    ref, tol = R.conv_bwd(n64(c["x"]), n64(c["w"]), n64(c["b"]), lens, n64(c["dy"]), n64(c["c0"]),
                          n64(c["dl"]) if carry else None, silu, io)
    for k in ("dx", "dweight") + (("dbias",) if silu else ()) + (("dconv0",) if carry else ()):
        R.check(k, n64(g[k]), ref[k], tol[k])
    assert (g["dbias"] is None) == (not silu) and (g["dconv0"] is None) == (not carry)
    for b, n in enumerate(R.lengths(lens, B, L)):
        assert not bits(g["dx"])[b, n:].any()
    if wide:
        assert (dx[..., D:] == 7).all()   # the other half of the buffer is left alone


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_large(io):
    """Work enough for the forward's long chunks and for several runs a workgroup in the backward, rows of every kind
    of length, an odd width."""
    import selective_state_space_scan_amd as ssm
    B, L, D, W = 5, 3500, 1001, 4
    lens = [3500, 3487, 12, 0, 1777]
    c = conv_inputs(io, B, L, D, W, 18)
    y, last = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], i32(lens), conv0=c["c0"])
    g = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], i32(lens), c["dy"], conv0=c["c0"], dconv_last=c["dl"])
    sync()
    a = (n64(c["x"]), n64(c["w"]), n64(c["b"]), lens)
    ry, rl, tol = R.conv_fwd(*a, n64(c["c0"]), True, io)
    R.check("y", n64(y), ry, tol)
    assert np.array_equal(n64(last), rl)
    ref, tol = R.conv_bwd(*a, n64(c["dy"]), n64(c["c0"]), n64(c["dl"]), True, io)
    for k in ref:
        R.check(k, n64(g[k]), ref[k], tol[k])
    again = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], i32(lens), c["dy"], conv0=c["c0"], dconv_last=c["dl"])
    assert all(np.array_equal(bits(g[k]), bits(again[k])) for k in g)   # run to run


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_every_form(io, W, silu):
    """Each number of taps with and without silu: the forward's long chunks and the backward's several runs a workgroup
    at an odd width, rows of every kind of length (2 runs of 13 steps a lane, 4 lanes, 3 workgroups a lane of
    the second pass and its exchanges, behind one another in a weight's sum), and one channel."""
    import selective_state_space_scan_amd as ssm
    B, L, D = 5, 3300, 1001
    lens = [3300, 3287, 12, 0, 1777]
    c = conv_inputs(io, B, L, D, W, 27, wide=True, bias=silu)
    y, last = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], i32(lens), silu=silu, conv0=c["c0"])
    g = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], i32(lens), c["dy"], silu=silu, conv0=c["c0"], dconv_last=c["dl"])
    sync()
    a = (n64(c["x"]), n64(c["w"]), n64(c["b"]), lens)
    ry, rl, tol = R.conv_fwd(*a, n64(c["c0"]), silu, io)
    R.check("y", n64(y), ry, tol)
    assert np.array_equal(n64(last), rl)
    ref, tol = R.conv_bwd(*a, n64(c["dy"]), n64(c["c0"]), n64(c["dl"]), silu, io)
    for k in ("dx", "dweight", "dconv0") + (("dbias",) if silu else ()):
        R.check(k, n64(g[k]), ref[k], tol[k])
    for b, n in enumerate(lens):
        assert not bits(y)[b, n:].any() and not bits(g["dx"])[b, n:].any()
    test_conv_fwd(io, 2, 30, 1, W, [30, 11], True, False, silu)
    test_conv_bwd(io, 2, 30, 1, W, [30, 11], True, False, silu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[37, 20, 52], None])
def test_conv_bwd_last_input_not_finite(io, lens):
    """An infinity or NaN as a row's last input meets one tap only: the steps behind it, which would bring it to the
    others, are not the row's."""
    import selective_state_space_scan_amd as ssm
    B, L, D, W = 3, 52, 70, 4
    c = conv_inputs(io, B, L, D, W, 19)
    ends = R.lengths(lens, B, L)
    bad, zero = c["x"].clone(), c["x"].clone()
    for b, v in enumerate((float("inf"), float("nan"), -float("inf"))):
        bad[b, ends[b] - 1, 4 + b], zero[b, ends[b] - 1, 4 + b] = v, 0.0
    g, ref = (ssm.causal_conv_bwd(x, c["w"], c["b"], i32(lens), c["dy"], silu=False, conv0=c["c0"])
              for x in (bad, zero))
    sync()
    for k in ("dx", "dbias", "dconv0"):   # without silu the inputs only reach the taps
        assert np.array_equal(bits(g[k]), bits(ref[k])), k
    got, want = n64(g["dweight"]), n64(ref["dweight"])
    dy = n64(c["dy"])
    for b, v in enumerate((np.inf, np.nan, -np.inf)):
        want[4 + b, W - 1] = v * dy[b, ends[b] - 1, 4 + b]
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_padding_reaches_nothing(io):
    """NaN, infinities and the type's lowest value past a row's end change no bit."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D, W = 4, 75, 40, 4
    lens = [75, 40, 1, 0]
    c = conv_inputs(io, B, L, D, W, 13)
    vl = i32(lens)

    def both(x, dy):
        y, last = ssm.causal_conv_fwd(x, c["w"], c["b"], vl, conv0=c["c0"])
        g = ssm.causal_conv_bwd(x, c["w"], c["b"], vl, dy, conv0=c["c0"], dconv_last=c["dl"])
        return [bits(t) for t in (y, last, g["dx"], g["dweight"], g["dbias"], g["dconv0"])]

    want = both(c["x"], c["dy"])
    for bad in (float("nan"), float("inf"), torch.finfo(_dt(io)).min):
        x, dy = c["x"].clone(), c["dy"].clone()
        for b, n in enumerate(lens):
            x[b, n:] = bad
            dy[b, n:] = bad
        for a, b in zip(both(x, dy), want):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_padding_with_infinite_weights(io, silu):
    """Steps past a row's end give +0, an infinity or NaN in taps or bias notwithstanding, in every chunk that a row's
    end may fall into."""
    import selective_state_space_scan_amd as ssm
    B, L, D, W = 6, 75, 40, 4
    lens = [75, 40, 13, 38, 1, 0]
    c = conv_inputs(io, B, L, D, W, 20)
    c["w"][3, 0], c["w"][7, 3], c["b"][9] = float("inf"), float("nan"), float("-inf")
    y, last = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], i32(lens), silu=silu, conv0=c["c0"])
    g = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], i32(lens), c["dy"], silu=silu, conv0=c["c0"], dconv_last=c["dl"])
    sync()
    for t in (y, g["dx"]):
        for b, n in enumerate(lens):
            assert not bits(t)[b, n:].any()
    # the other channels are those of finite weights
    ok = [d for d in range(D) if d not in (3, 7, 9)]
    f = conv_inputs(io, B, L, D, W, 20)
    r = ssm.causal_conv_bwd(f["x"], f["w"], f["b"], i32(lens), f["dy"], silu=silu, conv0=f["c0"], dconv_last=f["dl"])
    assert np.array_equal(bits(g["dx"])[..., ok], bits(r["dx"])[..., ok])
    assert np.array_equal(bits(g["dweight"])[ok], bits(r["dweight"])[ok])


def test_conv_infinite_and_nan_inputs_follow_the_formula():
    """Inside a row they spread over the W steps that see them and no further."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D = 1, 24, 8
    x = torch.ones((B, L, D), device=DEV)
    x[0, 10, 3] = float("nan")
    x[0, 10, 4] = float("inf")
    x[0, 10, 5] = -3e38
    w = torch.ones((D, 4), device=DEV)
    y, _ = ssm.causal_conv_fwd(x, w)
    sync()
    y = n64(y)[0]
    assert np.isnan(y[10:14, 3]).all() and np.isposinf(y[10:14, 4]).all() and (np.abs(y[10:14, 5]) == 0).all()
    keep = np.ones((L, D), bool)
    keep[10:14, 3:6] = False
    assert np.isfinite(y[keep]).all()


def test_silu_far_from_zero():
    """x = -110..110 through one tap: relative accuracy where sigmoid(x) is a normal fp32 number.  Below x = -87.3 it
    is less than 2^-126, and v_rcp_f32 returns 0 for a result (or an e^-x) out of fp32's normal range: sigmoid is off
    by at most 2^-126 there, x * sigmoid(x) by |x| 2^-126 (1.3e-36 at -110)."""
    import torch
    import selective_state_space_scan_amd as ssm
    v = torch.linspace(-110, 110, 4001, device=DEV)
    w = torch.tensor([[0.0, 1.0]], device=DEV)
    y, _ = ssm.causal_conv_fwd(v.view(1, -1, 1).contiguous(), w)
    sync()
    p = n64(v)
    ref = p / (1 + np.exp(-p))
    R.check("y", n64(y).ravel(), ref, 12 * R.U * np.abs(ref) + np.abs(p) * 2.0 ** -126)


def test_conv_time_major_views():
    """x, y, dy and dx as [L, B, D] buffers seen as [B, L, D]."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D, W = 3, 50, 24, 4
    c = conv_inputs("bf16", B, L, D, W, 14)
    tm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    y0, l0 = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], conv0=c["c0"])
    y1, l1 = ssm.causal_conv_fwd(tm(c["x"]), c["w"], c["b"], conv0=c["c0"], y=tm(torch.zeros_like(y0)))
    assert y1.stride() != y0.stride() and torch.equal(y0, y1) and torch.equal(l0, l1)
    g0 = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], None, c["dy"])
    g1 = ssm.causal_conv_bwd(tm(c["x"]), c["w"], c["b"], None, tm(c["dy"]), dx=tm(torch.zeros_like(y0)))
    for k in ("dx", "dweight", "dbias"):
        assert torch.equal(g0[k], g1[k]), k


def test_conv_repeated_inputs():
    """Inputs with stride 0 (one row for the whole batch, one gradient for every step)."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D, W = 4, 33, 16, 3
    c = conv_inputs("f32", B, L, D, W, 15)
    x, dy = c["x"][:1].expand(B, L, D), c["dy"][:, :1].expand(B, L, D)
    y0, _ = ssm.causal_conv_fwd(x, c["w"], c["b"])
    y1, _ = ssm.causal_conv_fwd(x.contiguous(), c["w"], c["b"])
    assert torch.equal(y0, y1)
    g0 = ssm.causal_conv_bwd(x, c["w"], c["b"], None, dy)
    g1 = ssm.causal_conv_bwd(x.contiguous(), c["w"], c["b"], None, dy.contiguous())
    for k in ("dx", "dweight", "dbias"):
        assert torch.equal(g0[k], g1[k]), k


@pytest.mark.parametrize("offset", [1, 3])
def test_conv_unaligned_views(offset):
    """Tensors that start inside their allocation, at no multiple of 16 bytes."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, L, D, W = 2, 40, 24, 4
    c = conv_inputs("bf16", B, L, D, W, 16)

    def off(t):
        flat = torch.zeros(t.numel() + offset, dtype=t.dtype, device=DEV)
        v = flat[offset:].view(t.shape)
        v.copy_(t)
        return v

    o = {k: off(v) for k, v in c.items()}
    y0, l0 = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], conv0=c["c0"])
    y1, l1 = ssm.causal_conv_fwd(o["x"], o["w"], o["b"], conv0=o["c0"], y=off(torch.zeros_like(y0)))
    assert torch.equal(y0, y1) and torch.equal(l0, l1)
    g0 = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], None, c["dy"], conv0=c["c0"], dconv_last=c["dl"])
    g1 = ssm.causal_conv_bwd(o["x"], o["w"], o["b"], None, o["dy"], conv0=o["c0"], dconv_last=o["dl"])
    for k in g0:
        assert torch.equal(g0[k], g1[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_empty(io):
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(17, io)
    w, b = g.normal(8, 4, io="f32"), g.normal(8, io="f32")
    c0, dl = g.normal(3, 3, 8), g.normal(3, 3, 8)
    x = torch.empty((3, 0, 8), dtype=_dt(io), device=DEV)
    y, last = ssm.causal_conv_fwd(x, w, b, conv0=c0)      # no steps: the carried inputs stay
    assert y.shape == x.shape and torch.equal(last, c0)
    _, last = ssm.causal_conv_fwd(x, w, b)
    assert (last == 0).all()
    r = ssm.causal_conv_bwd(x, w, b, None, x, conv0=c0, dconv_last=dl)
    assert torch.equal(r["dconv0"], dl) and (r["dweight"] == 0).all() and (r["dbias"] == 0).all()
    x = torch.empty((0, 5, 8), dtype=_dt(io), device=DEV)
    y, last = ssm.causal_conv_fwd(x, w, b)
    assert y.numel() == 0 and last.shape == (0, 3, 8)
    r = ssm.causal_conv_bwd(x, w, b, None, x)
    assert (r["dweight"] == 0).all() and (r["dbias"] == 0).all()
    x = torch.empty((2, 5, 0), dtype=_dt(io), device=DEV)
    y, last = ssm.causal_conv_fwd(x, w[:0], None)
    assert y.numel() == 0
    assert ssm.causal_conv_bwd(x, w[:0], None, None, x)["dweight"].shape == (0, 4)


# ---- single tokens -----------------------------------------------------------

@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("io,B,D,W,slots", [
    ("f32", 1, 64, 4, None), ("bf16", 3, 72, 4, None), ("bf16", 5, 13, 3, [6, 0, -1, 2, 5]),
    ("f32", 4, 7, 2, [7, 3, 8, 100]), ("bf16", 6, 2056, 4, [3, 1, 3, 0, 1, -7]), ("f32", 1, 1, 3, [0])])
def test_conv_step(io, B, D, W, slots, silu):
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(21, io)
    n = B if slots is None else 8
    cache = g.normal(n, W - 1, D)
    x, w, b = g.normal(B, 2 * D)[:, D:], g.normal(D, W, io="f32", scale=0.5), g.normal(D, io="f32") if silu else None
    new = torch.full_like(cache, 9.0)
    y = ssm.causal_conv_step(x, cache, w, b, silu=silu, slots=i32(slots), conv_last=new)
    inplace = cache.clone()
    y2 = ssm.causal_conv_step(x, inplace, w, b, silu=silu, slots=i32(slots))
    sync()
    live, seen = [], set()
    for i in range(B):
        s = i if slots is None else slots[i]
        if 0 <= s < n and s not in seen:
            live.append((i, s))
            seen.add(s)
    rows, at = [i for i, _ in live], [s for _, s in live]
    ry, rl, tol = R.conv_fwd(n64(x)[rows][:, None], n64(w), n64(b), None, n64(cache)[at], silu, io)
    R.check("y", n64(y)[rows], ry[:, 0], tol[:, 0])
    assert np.array_equal(n64(new)[at], rl)
    idle = [i for i in range(B) if i not in rows]
    rest = [s for s in range(n) if s not in seen]
    assert not bits(y)[idle].any() and (n64(new)[rest] == 9).all()
    assert torch.equal(y, y2) and torch.equal(inplace[at], new[at]) and torch.equal(inplace[rest], cache[rest])


STEP = [
    # io, B, D, N, slots, gate, skip, bias, clamp
    ("f32", 1, 64, 16, None, True, True, True, None),
    ("bf16", 3, 72, 16, None, False, True, False, (0.01, 0.5)),
    ("bf16", 5, 13, 32, [6, 0, -1, 2, 5], True, False, True, None),
    ("f32", 4, 7, 64, [7, 3, 8, 100], False, False, False, None),
    ("bf16", 6, 130, 64, [3, 1, 3, 0, 1, -7], True, True, True, (0.01, 0.5)),
    ("f32", 2, 1, 16, [1, 0], True, True, True, None),
]


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("io,B,D,N,slots,gate,skip,bias,clamp", STEP)
def test_scan_step(io, B, D, N, slots, gate, skip, bias, clamp, softplus):
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(22, io)
    n = B if slots is None else 8
    h = g.normal(n, D, N, io="f32")
    x = g.normal(B, 2 * D)[:, D:]
    delta = g.normal(B, D + 3, scale=0.5)[:, 3:] if softplus else g.normal(B, D).abs() * 0.3
    bc = g.normal(B, 2 * N + 5)
    Bm, Cm = bc[:, 5:N + 5], bc[:, N + 5:]
    A_log = g.normal(D, N, io="f32", shift=1.0)
    Dk = g.normal(D, io="f32") if skip else None
    db = g.normal(D, io="f32") if bias and softplus else None
    z = g.normal(B, 3 * D)[:, D:2 * D] if gate else None
    kw = dict(slots=i32(slots), delta_softplus=softplus, delta_clamp=clamp, delta_bias=db, z=z)
    new = torch.full_like(h, 9.0)
    wide = torch.full((B, 2 * D), 5.0, dtype=_dt(io), device=DEV)
    y = ssm.selective_scan_step(x, delta, A_log, Bm, Cm, Dk, h, h_last=new, y=wide[:, :D], **kw)
    inplace = h.clone()
    y2 = ssm.selective_scan_step(x, delta, A_log, Bm, Cm, Dk, inplace, **kw)
    sync()
    live, seen = [], set()
    for i in range(B):
        s = i if slots is None else slots[i]
        if 0 <= s < n and s not in seen:
            live.append((i, s))
            seen.add(s)
    rows, at = [i for i, _ in live], [s for _, s in live]
    clamp64 = None if clamp is None else tuple(float(np.float32(v)) for v in clamp)
    ry, rh, ty, th = R.scan_step(n64(x)[rows], n64(delta)[rows], n64(A_log), n64(Bm)[rows], n64(Cm)[rows], n64(Dk),
                                 n64(h)[at], n64(db), None if z is None else n64(z)[rows], softplus, clamp64, io)
    R.check("h_last", n64(new)[at], rh, th)
    R.check("y", n64(y)[rows], ry, ty)
    idle = [i for i in range(B) if i not in rows]
    rest = [s for s in range(n) if s not in seen]
    assert not bits(y)[idle].any() and (n64(new)[rest] == 9).all() and (wide[:, D:] == 5).all()
    assert torch.equal(y, y2) and torch.equal(inplace[at], new[at]) and torch.equal(inplace[rest], h[rest])


@pytest.mark.parametrize("softplus", [True, False])
def test_clip_of_a_delta_that_is_not_finite(softplus):
    """The step's clip is the scan's: NaN becomes the lower bound, infinities the bounds; without a clip NaN spreads."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, D, N = 3, 32, 16
    lo, hi = 0.125, 0.5
    g = Gen(25, "f32")
    x, bm, cm, A, h = g.normal(B, D), g.normal(B, N), g.normal(B, N), g.normal(D, N), g.normal(B, D, N)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV)[:, None].expand(B, D).contiguous()
    bound = torch.tensor([lo, hi, lo], device=DEV)[:, None].expand(B, D).contiguous()
    want_h, got_h = h.clone(), h.clone()
    want = ssm.selective_scan_step(x, bound, A, bm, cm, None, want_h, delta_softplus=False)
    got = ssm.selective_scan_step(x, bad, A, bm, cm, None, got_h, delta_softplus=softplus, delta_clamp=(lo, hi))
    assert torch.equal(got, want) and torch.equal(got_h, want_h)
    seq = [t[:, None].contiguous() for t in (x, bad, bound, bm, cm)]
    y0, h0 = ssm.selective_scan_fwd(seq[0], seq[2], A, seq[3], seq[4], h0=h, delta_softplus=False)
    y1, h1 = ssm.selective_scan_fwd(seq[0], seq[1], A, seq[3], seq[4], h0=h, delta_softplus=softplus,
                                    delta_clamp=(lo, hi))
    assert torch.equal(y1, y0) and torch.equal(h1, h0)
    y = ssm.selective_scan_step(x, bad, A, bm, cm, None, got_h, delta_softplus=softplus)
    assert torch.isnan(y[0]).all() and torch.isnan(got_h[0]).all()


@pytest.mark.parametrize("gate,skip,bias,clamp", [(True, True, True, (0.01, 0.5)), (False, False, True, None),
                                                  (True, False, False, (0.05, 0.4))])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_step_two_rows_a_workgroup(io, N, gate, skip, bias, clamp):
    """257 rows of 16 workgroups each with slots take two rows a workgroup, the last alone: idle rows first and second
    of a pair, slots repeated within a pair, in a later one and by the last row."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, D, n = 257, 15 * (1024 // N) + 7, 300
    g = Gen(26, io)
    h = g.normal(n, D, N, io="f32")
    x, delta, z = g.normal(B, 2 * D)[:, D:], g.normal(B, D, scale=0.5), g.normal(B, D) if gate else None
    bc = g.normal(B, 2 * N)
    Bm, Cm, A_log = bc[:, :N], bc[:, N:], g.normal(D, N, io="f32", shift=1.0)
    Dk, db = g.normal(D, io="f32") if skip else None, g.normal(D, io="f32") if bias else None
    slots = torch.randperm(n, generator=g.g)[:B].tolist()
    slots[2], slots[101], slots[150] = -1, n, -2**31
    slots[5], slots[20], slots[77], slots[256] = slots[4], slots[7], slots[30], slots[0]
    new = torch.full_like(h, 9.0)
    kw = dict(slots=i32(slots), delta_clamp=clamp, delta_bias=db, z=z)
    y = ssm.selective_scan_step(x, delta, A_log, Bm, Cm, Dk, h, h_last=new, **kw)
    inplace = h.clone()
    y2 = ssm.selective_scan_step(x, delta, A_log, Bm, Cm, Dk, inplace, **kw)
    sync()
    idle = [2, 101, 150, 5, 20, 77, 256]
    rows = [b for b in range(B) if b not in idle]
    at = [slots[b] for b in rows]
    rest = [s for s in range(n) if s not in at]
    clamp64 = None if clamp is None else tuple(float(np.float32(v)) for v in clamp)
    ry, rh, ty, th = R.scan_step(n64(x)[rows], n64(delta)[rows], n64(A_log), n64(Bm)[rows], n64(Cm)[rows], n64(Dk),
                                 n64(h)[at], n64(db), None if z is None else n64(z)[rows], True, clamp64, io)
    R.check("h_last", n64(new)[at], rh, th)
    R.check("y", n64(y)[rows], ry, ty)
    assert not bits(y)[idle].any() and (n64(new)[rest] == 9).all()
    assert torch.equal(y, y2) and torch.equal(inplace[at], new[at]) and torch.equal(inplace[rest], h[rest])


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_every_form_of_a_step(io, silu):
    """The taps and state counts that the lists above leave out for a type."""
    for W in (2, 3, 4):
        test_conv_step(io, 3, 24, W, [1, -1, 4], silu)
    for N in (16, 32, 64):
        test_scan_step(io, 2, 24, N, None, silu, True, True, None, True)


def test_idle_rows_read_nothing():
    """What an idle row's inputs hold, NaN included, reaches no output; an empty cache leaves every row idle."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, D, N, W = 3, 40, 16, 4
    g = Gen(23, "bf16")
    x, dl, bm = g.normal(B, D), g.normal(B, D), g.normal(B, N)
    for t in (x, dl, bm):
        t[1] = float("nan")
    A, w = g.normal(D, N, io="f32"), g.normal(D, W, io="f32")
    h, c = g.normal(4, D, N, io="f32"), g.normal(4, W - 1, D)
    slots = i32([2, -1, 0])
    y = ssm.selective_scan_step(x, dl, A, bm, bm, None, h, slots=slots)
    yc = ssm.causal_conv_step(x, c, w, slots=slots)
    assert torch.isfinite(y).all() and torch.isfinite(h).all() and torch.isfinite(yc).all() and torch.isfinite(c).all()
    y = ssm.selective_scan_step(x, dl, A, bm, bm, None, h[:0], slots=slots)
    yc = ssm.causal_conv_step(x, c[:0], w, slots=slots)
    assert (y == 0).all() and (yc == 0).all()
    # no rows
    assert ssm.selective_scan_step(x[:0], dl[:0], A, bm[:0], bm[:0], None, h, slots=slots[:0]).shape == (0, D)
    assert ssm.causal_conv_step(x[:0], c, w, slots=slots[:0]).shape == (0, D)


@pytest.mark.parametrize("D", [24, 330])
def test_many_rows_with_repeated_slots(D):
    """More rows than a wave's lanes, every slot named three times and one a fourth: the first of each takes the step.
    The wider one runs two rows a workgroup, the last alone."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, N, W = 901, 16, 4
    g = Gen(24, "f32")
    x, dl, bm, cm = g.normal(B, D), g.normal(B, D), g.normal(B, N), g.normal(B, N)
    A, w = g.normal(D, N, io="f32"), g.normal(D, W, io="f32")
    h, c = g.normal(300, D, N), g.normal(300, W - 1, D)
    order = torch.cat([torch.randperm(300, generator=g.g) for _ in range(3)] + [torch.tensor([7])]).to(DEV, torch.int32)
    first = 300   # each permutation names every slot once
    h1, c1 = h.clone(), c.clone()
    y = ssm.selective_scan_step(x, dl, A, bm, cm, None, h1, slots=order)
    yc = ssm.causal_conv_step(x, c1, w, slots=order)
    h2, c2 = h.clone(), c.clone()
    y2 = ssm.selective_scan_step(x[:first], dl[:first], A, bm[:first], cm[:first], None, h2, slots=order[:first])
    yc2 = ssm.causal_conv_step(x[:first], c2, w, slots=order[:first])
    assert torch.equal(h1, h2) and torch.equal(c1, c2) and torch.equal(y[:first], y2) and torch.equal(yc[:first], yc2)
    assert (y[first:] == 0).all() and (yc[first:] == 0).all()


# ---- norms -------------------------------------------------------------------

NORM = [
    # io, rio, B, L, D, lens
    ("f32", None, 1, 1, 1, None), ("f32", "f32", 3, 5, 7, [5, 0, 2]), ("bf16", None, 2, 9, 64, None),
    ("bf16", "f32", 2, 6, 72, [6, 3]), ("bf16", "bf16", 1, 5, 513, None), ("f32", None, 1, 4, 1000, None),
    ("bf16", "f32", 2, 3, 1030, [1, -1]), ("f32", "f32", 1, 3, 2049, None), ("bf16", "bf16", 1, 3, 4100, [99]),
    ("bf16", "f32", 1, 2, 8192, None), ("f32", None, 1, 2, 8200, None), ("bf16", None, 1, 2, 16384, None),
    ("f32", "f32", 1, 3, 16383, [2]),
]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("io,rio,B,L,D,lens", NORM)
def test_norm_fwd(io, rio, B, L, D, lens, rms):
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(31, io)
    x, w = g.normal(B, L, D), g.normal(D, io="f32", scale=0.2, shift=1.0)
    b = None if rms else g.normal(D, io="f32")
    res = None if rio is None else g.normal(B, L, D, io=rio, shift=0.7)
    y, v, mean, rstd = ssm.layer_norm_fwd(x, w, b, i32(lens), residual=res, rms=rms, return_stats=True)
    sync()
    flat = lambda t: None if t is None else n64(t).reshape(B * L, D)  # noqa: E731
    (ry, rv, rm, rr), (ty, tv, tm, tr) = R.norm_fwd(flat(x), n64(w), n64(b), flat(res), 1e-5, rms, io, rio or io)
    live = np.zeros((B, L), bool)
    for i, n in enumerate(R.lengths(lens, B, L)):
        live[i, :n] = True
    live = live.ravel()
    R.check("y", flat(y)[live], ry[live], ty[live])
    R.check("rstd", n64(rstd).ravel()[live], rr[live], tr[live])
    assert not bits(y).reshape(-1, D)[~live].any() and not bits(rstd).ravel()[~live].any()
    assert (mean is None) == rms and (v is None) == (res is None)
    if not rms:
        R.check("mean", n64(mean).ravel()[live], rm[live], tm[live])
        assert not bits(mean).ravel()[~live].any()
    if v is not None:
        R.check("residual_out", flat(v)[live], rv[live], tv[live])
        assert not bits(v).reshape(-1, D)[~live].any()
        inplace = res.clone()
        y2, v2 = ssm.layer_norm_fwd(x, w, b, i32(lens), residual=inplace, residual_out=inplace, rms=rms)
        assert v2 is inplace and torch.equal(inplace, v) and torch.equal(y2, y)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("io,rio,B,L,D,lens", NORM)
def test_norm_bwd(io, rio, B, L, D, lens, rms):
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(32, io)
    v, w = g.normal(B, L, D, io=rio or io, shift=0.7, scale=2.0), g.normal(D, io="f32", scale=0.2, shift=1.0)
    dy = g.normal(B, L, D)
    dr = None if rio is None else g.normal(B, L, D, io=rio)
    v64 = n64(v)
    m64 = np.zeros((B, L)) if rms else v64.mean(-1)
    rstd = torch.tensor(1 / np.sqrt(((v64 - m64[..., None]) ** 2).mean(-1) + 1e-5), dtype=torch.float32, device=DEV)
    mean = None if rms else torch.tensor(m64, dtype=torch.float32, device=DEV)
    out = ssm.layer_norm_bwd(dy, v, w, mean, rstd, i32(lens), dresidual_out=dr, with_bias=not rms)
    sync()
    live = np.zeros((B, L), bool)
    for i, n in enumerate(R.lengths(lens, B, L)):
        live[i, :n] = True
    live = live.ravel()
    flat = lambda t: n64(t).reshape(B * L, D)[live]  # noqa: E731
    ref, tol = R.norm_bwd(flat(dy), flat(v), n64(w), None if rms else n64(mean).ravel()[live],
                          n64(rstd).ravel()[live], None if dr is None else flat(dr), io, rio or io)
    R.check("dx", flat(out["dx"]), ref["dx"], tol["dx"])
    R.check("dweight", n64(out["dweight"]), ref["dweight"], tol["dweight"])
    assert not bits(out["dx"]).reshape(-1, D)[~live].any()
    assert (out["dbias"] is None) == rms and (out["dresidual"] is None) == (dr is None)
    if not rms:
        R.check("dbias", n64(out["dbias"]), ref["dbias"], tol["dbias"])
    if dr is not None:
        assert out["dresidual"].dtype == v.dtype and (out["dresidual"] is out["dx"]) == (io == rio)
        R.check("dresidual", flat(out["dresidual"]), ref["dresidual"], tol["dresidual"])


NORM_TYPES = [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [300, 600, 1024, 1500, 3000, 6000, 12000])
@pytest.mark.parametrize("io,rio", NORM_TYPES)
def test_norm_every_row_width(io, rio, D, rms):
    """64 to 1024 lanes a row, 8 and 16 elements a lane, each with rows past the valid length."""
    test_norm_fwd(io, rio, 2, 5, D, [5, 3], rms)
    test_norm_bwd(io, rio, 2, 5, D, [5, 3], rms)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D,L", [(40, 4001), (700, 2001), (1500, 1001), (3000, 251), (6000, 251), (9000, 251)])
@pytest.mark.parametrize("io,rio", NORM_TYPES)
def test_norm_many_rows_of_every_width(io, rio, D, L, rms):
    """Several rows a workgroup of the backward (at most 1280 of them, 256 where a row takes more than 256 lanes, of
    256 lanes): sums over rows in registers and over a row in LDS, one row after the other, some past their valid
    length.  The weight gradients' sums: at most 4 rows a lane, 4 lanes of a workgroup, 20 workgroups a lane of the
    second pass, its 8 exchanges; the row's: 16 elements, 6 exchanges, 16 waves."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(39, io)
    B, lens = 3, [L, L // 2, L - 1]
    x, dy = g.normal(B, L, D, shift=0.5), g.normal(B, L, D)
    w, b = g.normal(D, io="f32", scale=0.2, shift=1.0), g.normal(D, io="f32")
    res = None if rio is None else g.normal(B, L, D, io=rio)
    y, v, mean, rstd = ssm.layer_norm_fwd(x, w, b, i32(lens), residual=res, rms=rms, return_stats=True)
    out = ssm.layer_norm_bwd(dy, x if v is None else v, w, mean, rstd, i32(lens), dresidual_out=res)
    sync()
    live = np.concatenate([np.arange(L) < n for n in lens])
    flat = lambda t: None if t is None else n64(t).reshape(-1, D)[live]  # noqa: E731
    per_row = lambda t: None if t is None else n64(t).ravel()[live]  # noqa: E731
    (ry, rv, rm, rr), (ty, tv, tm, tr) = R.norm_fwd(flat(x), n64(w), n64(b), flat(res), 1e-5, rms, io, rio or io)
    R.check("y", flat(y), ry, ty)
    R.check("rstd", per_row(rstd), rr, tr)
    if v is not None:
        R.check("residual_out", flat(v), rv, tv)
    ref, tol = R.norm_bwd(flat(dy), flat(x if v is None else v), n64(w), per_row(mean), per_row(rstd), flat(res), io,
                          rio or io)
    for k in ("dx", "dweight", "dbias"):
        R.check(k, flat(out[k]) if k == "dx" else n64(out[k]), ref[k], tol[k])
    if res is not None:
        R.check("dresidual", flat(out["dresidual"]), ref["dresidual"], tol["dresidual"])
    for t in (y, out["dx"]) + (() if v is None else (v, out["dresidual"])):
        assert not bits(t).reshape(-1, D)[~live].any()
    again = ssm.layer_norm_bwd(dy, x if v is None else v, w, mean, rstd, i32(lens), dresidual_out=res)
    assert all(torch.equal(out[k], again[k]) for k in ("dx", "dweight", "dbias"))


def test_norm_many_rows():
    """More rows than the backward has workgroups: the weights' sums over several rows a lane."""
    import selective_state_space_scan_amd as ssm
    import torch
    g = Gen(33, "f32")
    rows, D = 9001, 40
    x, dy, w, b = g.normal(rows, D), g.normal(rows, D), g.normal(D), g.normal(D)
    y, _, mean, rstd = ssm.layer_norm_fwd(x, w, b, return_stats=True)
    out = ssm.layer_norm_bwd(dy, x, w, mean, rstd)
    (ry, _, _, _), (ty, _, _, _) = R.norm_fwd(n64(x), n64(w), n64(b))
    R.check("y", n64(y), ry, ty)
    ref, tol = R.norm_bwd(n64(dy), n64(x), n64(w), n64(mean), n64(rstd))
    for k in ("dx", "dweight", "dbias"):
        R.check(k, n64(out[k]), ref[k], tol[k])
    again = ssm.layer_norm_bwd(dy, x, w, mean, rstd)
    assert all(torch.equal(out[k], again[k]) for k in ("dx", "dweight", "dbias"))   # run to run


def test_norm_rows_far_from_zero_and_constant_rows():
    """A mean 10^4 times the spread costs only what the inputs' own rounding costs; a constant row gives the bias."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(34, "f32")
    x = g.normal(6, 700, shift=1e4)
    x[3] = 17.0
    x[4] = -3e4
    w, b = g.normal(700, shift=1.0), g.normal(700)
    y, _, mean, rstd = ssm.layer_norm_fwd(x, w, b, return_stats=True)
    sync()
    (ry, _, rm, rr), (ty, _, tm, tr) = R.norm_fwd(n64(x), n64(w), n64(b))
    R.check("y", n64(y), ry, ty)
    R.check("mean", n64(mean), rm, tm)
    R.check("rstd", n64(rstd), rr, tr)
    assert torch.equal(y[3], b) and torch.equal(y[4], b)


@pytest.mark.parametrize("D", [7, 700, 5001])
def test_norm_constant_rows_far_from_zero(D):
    """The variance of a constant row is what rounding leaves of zero: it must not come out negative."""
    import torch
    import selective_state_space_scan_amd as ssm
    x = torch.tensor([1e9, -3.3e9, 7.7e10, 1.1e12, 3e5, 123456.7], device=DEV)[:, None].expand(6, D).contiguous()
    w = torch.ones(D, device=DEV)
    y, _, mean, rstd = ssm.layer_norm_fwd(x, w, return_stats=True)
    sync()
    (ry, _, rm, _), (ty, _, tm, _) = R.norm_fwd(n64(x), n64(w), None)
    R.check("y", n64(y), ry, ty)
    R.check("mean", n64(mean), rm, tm)
    assert torch.isfinite(rstd).all() and (rstd > 0).all()


def test_norm_bad_rows_stay_alone():
    """NaN or infinity in a row spoils that row and, in the backward, the weights' sums, nothing else; past a
    row's valid length nothing."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(35, "bf16")
    x, res = g.normal(2, 4, 96), g.normal(2, 4, 96, io="f32")
    w, dy = g.normal(96, io="f32"), g.normal(2, 4, 96)
    y0, v0 = ssm.layer_norm_fwd(x, w, residual=res)
    bad = x.clone()
    bad[0, 1, 5] = float("nan")
    bad[1, 2, 7] = float("inf")
    y, _ = ssm.layer_norm_fwd(bad, w, residual=res)
    ok = torch.ones((2, 4), dtype=torch.bool, device=DEV)
    ok[0, 1] = ok[1, 2] = False
    assert torch.equal(y[ok], y0[ok]) and torch.isnan(y[~ok]).all(1).all()
    vl = i32([1, 2])
    for f in (x, bad):
        outs = [*ssm.layer_norm_fwd(f, w, None, vl, residual=res, return_stats=True)]
        b = ssm.layer_norm_bwd(f, v0, w, outs[2], outs[3], vl, dresidual_out=res)
        outs += [b[k] for k in ("dx", "dresidual", "dweight", "dbias")]
        if f is x:
            want = outs
        assert all(np.array_equal(bits(p), bits(q)) for p, q in zip(outs, want))


@pytest.mark.parametrize("io,rio", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("D", [7, 200, 1001, 2050, 9001])
def test_norm_bwd_of_large_means(D, io, rio):
    """Rows that are constant and so large that mean * rstd leaves fp32's range: v - mean is 0 in every element, and
    the places past a row's end that widths leave in the last lanes have no say."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(37, io)
    v = torch.tensor([3e36, -1e37, 2.5], device=DEV).to(_dt(rio))[:, None].expand(3, D).contiguous()
    mean, rstd = v[:, 0].float().contiguous(), torch.full((3,), 1e-5 ** -0.5, device=DEV)
    dy, w, dr = g.normal(3, D), g.normal(D, io="f32"), g.normal(3, D, io=rio)
    out = ssm.layer_norm_bwd(dy, v, w, mean, rstd, dresidual_out=dr)
    sync()
    ref, tol = R.norm_bwd(n64(dy), n64(v), n64(w), n64(mean), n64(rstd), n64(dr), io, rio)
    for k in ("dx", "dresidual", "dweight", "dbias"):
        R.check(k, n64(out[k]), ref[k], tol[k])


@pytest.mark.parametrize("io,rio", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("D", [40, 1030])
def test_norm_padding_with_infinite_weights(D, io, rio):
    """Rows past the valid length give +0 in every output, an infinity or NaN in weight or bias notwithstanding."""
    import selective_state_space_scan_amd as ssm
    g = Gen(38, io)
    B, L = 3, 5
    lens = [2, 0, 4]
    x, res, w, b = g.normal(B, L, D), g.normal(B, L, D, io=rio), g.normal(D, io="f32"), g.normal(D, io="f32")
    w[3], w[-1], b[5] = float("inf"), float("nan"), float("-inf")
    y, v, mean, rstd = ssm.layer_norm_fwd(x, w, b, i32(lens), residual=res, return_stats=True)
    out = ssm.layer_norm_bwd(x, v, w, mean, rstd, i32(lens), dresidual_out=res)
    sync()
    for t in (y, v, mean, rstd, out["dx"], out["dresidual"]):
        for i, n in enumerate(lens):
            assert not bits(t)[i, n:].any()
    assert np.isfinite(n64(out["dweight"])).all() and np.isfinite(n64(out["dbias"])).all()


def test_norm_empty():
    import torch
    import selective_state_space_scan_amd as ssm
    w = torch.ones(16, device=DEV)
    x = torch.empty((0, 16), device=DEV)
    y, v = ssm.layer_norm_fwd(x, w)
    assert y.shape == (0, 16) and v is None
    out = ssm.layer_norm_bwd(x, x, w, torch.empty(0, device=DEV), torch.empty(0, device=DEV))
    assert (out["dweight"] == 0).all() and (out["dbias"] == 0).all()
    x = torch.empty((4, 0), device=DEV)
    y, _ = ssm.layer_norm_fwd(x, w[:0])
    assert y.shape == (4, 0)


def test_norm_statistics_of_no_elements():
    """Rows of no elements: mean 0 and rstd 1 / sqrt(eps), padded rows 0, all written."""
    import torch
    import selective_state_space_scan_amd as ssm
    keep = [torch.full((3, 4), 7.0, device=DEV) for _ in range(2)]
    del keep   # what the allocator hands out next holds something
    x, w = torch.empty((3, 4, 0), device=DEV), torch.empty(0, device=DEV)
    y, _, mean, rstd = ssm.layer_norm_fwd(x, w, None, i32([4, 0, 2]), eps=0.25, return_stats=True)
    assert y.shape == (3, 4, 0) and not mean.any()
    assert rstd.tolist() == [[2.0] * 4, [0.0] * 4, [2.0] * 2 + [0.0] * 2]
    _, _, none, rstd = ssm.layer_norm_fwd(x, w, None, i32([4, 0, 2]), eps=0.25, rms=True, return_stats=True)
    assert none is None and rstd.tolist() == [[2.0] * 4, [0.0] * 4, [2.0] * 2 + [0.0] * 2]


def test_norm_starts_a_residual_stream():
    """residual_out without residual: x itself, in the stream's own type."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(36, "bf16")
    x, w = g.normal(5, 72), g.normal(72, io="f32")
    v = torch.empty((5, 72), dtype=torch.float32, device=DEV)
    y, r = ssm.layer_norm_fwd(x, w, residual_out=v)
    y0, none = ssm.layer_norm_fwd(x, w)
    assert r is v and torch.equal(v, x.float()) and torch.equal(y, y0) and none is None


# ---- streams, offsets, refusals -----------------------------------------------

def _all_ops(seed=41):
    """One call of every operator: a list of (name, function of a stream, outputs as tensors)."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(seed, "bf16")
    B, L, D, N, W = 3, 90, 136, 16, 4
    c = conv_inputs("bf16", B, L, D, W, seed)
    vl = i32([90, 7, 55])
    x, dl, bm, cm = g.normal(B, D), g.normal(B, D), g.normal(B, N), g.normal(B, N)
    A, h, cache, sl = g.normal(D, N, io="f32"), g.normal(8, D, N, io="f32"), g.normal(8, W - 1, D), i32([5, -1, 2])
    xn, res, w, b = g.normal(200, D), g.normal(200, D, io="f32"), g.normal(D, io="f32"), g.normal(D, io="f32")
    mean, rstd = res.mean(1), torch.rsqrt(res.var(1, unbiased=False) + 1e-5)
    h_last, c_last = torch.zeros_like(h), torch.zeros_like(cache)
    sync()

    def flat(r):
        return [t for t in (r.values() if isinstance(r, dict) else r) if t is not None]

    return [
        ("conv_fwd", lambda s=None: flat(ssm.causal_conv_fwd(c["x"], c["w"], c["b"], vl, conv0=c["c0"], stream=s))),
        ("conv_bwd", lambda s=None: flat(ssm.causal_conv_bwd(c["x"], c["w"], c["b"], vl, c["dy"], conv0=c["c0"],
                                                            dconv_last=c["dl"], stream=s))),
        ("conv_step", lambda s=None: [ssm.causal_conv_step(x, cache, c["w"], c["b"], slots=sl, conv_last=c_last,
                                                          stream=s), c_last]),
        ("scan_step", lambda s=None: [ssm.selective_scan_step(x, dl, A, bm, cm, b, h, slots=sl, h_last=h_last, z=x,
                                                             stream=s), h_last]),
        ("norm_fwd", lambda s=None: flat(ssm.layer_norm_fwd(xn, w, b, residual=res, return_stats=True, stream=s))),
        ("norm_bwd", lambda s=None: flat(ssm.layer_norm_bwd(xn, res, w, mean, rstd, dresidual_out=res, stream=s))),
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
    sets = [_all_ops(41), _all_ops(42)]
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


def test_graph_replays():
    """Every operator captured, replayed on changed inputs with eager work between, equals the eager call."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(43, "bf16")
    B, L, D, N, W = 2, 300, 136, 16, 4
    st = dict(x=g.normal(B, L, D), dy=g.normal(B, L, D), vl=i32([300, 11]), c0=g.normal(B, W - 1, D),
              t=g.normal(B, D), bm=g.normal(B, N), h=g.normal(4, D, N, io="f32"), cache=g.normal(4, W - 1, D),
              sl=i32([3, 1]), res=g.normal(B * L, D, io="f32"))
    w, b, A, nw = g.normal(D, W, io="f32"), g.normal(D, io="f32"), g.normal(D, N, io="f32"), g.normal(D, io="f32")
    outs = dict(h=torch.zeros_like(st["h"]), c=torch.zeros_like(st["cache"]))

    def run():
        y, last = ssm.causal_conv_fwd(st["x"], w, b, st["vl"], conv0=st["c0"])
        cb = ssm.causal_conv_bwd(st["x"], w, b, st["vl"], st["dy"], conv0=st["c0"], dconv_last=last)
        yc = ssm.causal_conv_step(st["t"], st["cache"], w, b, slots=st["sl"], conv_last=outs["c"])
        ys = ssm.selective_scan_step(yc, st["t"], A, st["bm"], st["bm"], b, st["h"], slots=st["sl"], h_last=outs["h"])
        yn, v, m, r = ssm.layer_norm_fwd(y.view(B * L, D), nw, b, residual=st["res"], return_stats=True)
        nb = ssm.layer_norm_bwd(yn, v, nw, m, r, dresidual_out=st["res"])
        return [y, last, *cb.values(), yc, ys, outs["c"], outs["h"], yn, v, m, r, *nb.values()]

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
    for k in range(4):
        for name in ("x", "dy", "c0", "t", "bm", "res"):
            st[name].copy_(torch.randn(st[name].shape, generator=g.g).to(st[name]))
        st["vl"].copy_(i32([300 - 100 * k, 11 * k]))
        st["sl"].copy_(i32([k, (k + 1) % 4 if k != 2 else -1]))
        outs["c"].zero_()
        outs["h"].zero_()
        graph.replay()
        sync()
        got = [t.clone() for t in static]
        outs["c"].zero_()
        outs["h"].zero_()
        want = run()
        sync()
        for i, (a, e) in enumerate(zip(got, want)):
            assert torch.equal(a, e), (k, i)


def test_two_graphs_of_the_backward():
    """Two captured backward passes, replayed at once on two streams: each has its own scratch."""
    import torch
    import selective_state_space_scan_amd as ssm
    sets = [conv_inputs("bf16", 2, 700, 136, 4, s) for s in (51, 52)]
    nw = torch.ones(136, device=DEV)
    graphs, static, want = [], [], []

    def run(c):
        g = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], None, c["dy"])
        rows = c["x"].view(-1, 136)
        _, _, m, r = ssm.layer_norm_fwd(rows, nw, return_stats=True)
        n = ssm.layer_norm_bwd(c["dy"].view(-1, 136), rows, nw, m, r)
        return [g["dx"], g["dweight"], g["dbias"], n["dx"], n["dweight"], n["dbias"]]

    for c in sets:
        want.append([t.clone() for t in run(c)])
        sync()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            static.append(run(c))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for t in static[0] + static[1]:
            t.zero_()
        sync()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        sync()
        for got, w in zip(static, want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_offsets_past_32_bits():
    """A cache and sequences of more than 2^32 bytes (and 2^31 elements): the last rows are as good as the first."""
    import torch
    import selective_state_space_scan_amd as ssm
    D, N, W = 2048, 16, 4
    g = Gen(61, "bf16")
    n = 2**31 // (D * N) + 9
    h = torch.zeros((n, D, N), device=DEV)
    x, dl, bm, A = g.normal(2, D), g.normal(2, D), g.normal(2, N), g.normal(D, N, io="f32")
    st = g.normal(2, D, N, io="f32")
    sl = i32([n - 1, 0])
    h[n - 1], h[0] = st[0], st[1]
    y = ssm.selective_scan_step(x, dl, A, bm, bm, None, h, slots=sl)
    y2 = ssm.selective_scan_step(x, dl, A, bm, bm, None, st)
    assert torch.equal(y, y2) and torch.equal(h[n - 1], st[0]) and torch.equal(h[0], st[1])
    assert not h[1:9].any() and not h[n - 9:n - 1].any()
    del h
    n = 2**31 // (D * (W - 1)) + 9
    cache = torch.zeros((n, W - 1, D), dtype=torch.bfloat16, device=DEV)
    w, cs = g.normal(D, W, io="f32"), g.normal(2, W - 1, D)
    cache[n - 1], cache[0] = cs[0], cs[1]
    sl = i32([n - 1, 0])
    y = ssm.causal_conv_step(x, cache, w, slots=sl)
    y2 = ssm.causal_conv_step(x, cs, w)
    assert torch.equal(y, y2) and torch.equal(cache[n - 1], cs[0]) and torch.equal(cache[0], cs[1])
    del cache
    # one sequence of 2^31 elements and a bit, compared at its end with a short run that carries on
    L = 2**31 // D + 100
    x = torch.empty((1, L, D), dtype=torch.bfloat16, device=DEV)
    x.view(torch.int16).random_(0x3f00, 0x3fff)   # 0.5 to 2
    y, last = ssm.causal_conv_fwd(x, w)
    tail, lt = ssm.causal_conv_fwd(x[:, L - 200:], w, conv0=x[:, L - 203:L - 200].contiguous())
    assert torch.equal(y[:, L - 200:], tail) and torch.equal(last, lt)
    g = ssm.causal_conv_bwd(x, w, None, None, y)
    gt = ssm.causal_conv_bwd(x[:, L - 200:], w, None, None, y[:, L - 200:], conv0=x[:, L - 203:L - 200].contiguous())
    assert torch.equal(g["dx"][:, L - 197:], gt["dx"][:, 3:])
    del g, gt, y
    rows = x.view(L, D)
    nw = torch.ones(D, device=DEV)
    y, _, m, r = ssm.layer_norm_fwd(rows, nw, return_stats=True)
    yt, _, mt, rt = ssm.layer_norm_fwd(rows[L - 50:], nw, return_stats=True)
    assert torch.equal(y[L - 50:], yt) and torch.equal(m[L - 50:], mt) and torch.equal(r[L - 50:], rt)
    g = ssm.layer_norm_bwd(y, rows, nw, m, r)
    gt = ssm.layer_norm_bwd(yt, rows[L - 50:], nw, mt, rt)
    assert torch.equal(g["dx"][L - 50:], gt["dx"])


def test_given_outputs_and_scratch():
    """Outputs and scratch that the caller owns are the ones written and returned."""
    import torch
    import selective_state_space_scan_amd as ssm
    c = conv_inputs("bf16", 2, 60, 24, 4, 62)
    y0, l0 = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], conv0=c["c0"])
    y, last = torch.zeros_like(y0), torch.zeros_like(l0)
    r = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], conv0=c["c0"], y=y, conv_last=last, return_conv_last=False)
    assert r[0] is y and r[1] is last and torch.equal(y, y0) and torch.equal(last, l0)
    y1, none = ssm.causal_conv_fwd(c["x"], c["w"], c["b"], conv0=c["c0"], return_conv_last=False)
    assert none is None and torch.equal(y1, y0)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)   # NaN where read before written
    g0 = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], None, c["dy"])
    g1 = ssm.causal_conv_bwd(c["x"], c["w"], c["b"], None, c["dy"], dx=y, workspace=ws)
    assert g1["dx"] is y and all(torch.equal(g0[k], g1[k]) for k in ("dx", "dweight", "dbias"))
    g = Gen(63, "bf16")
    x, res, w = g.normal(70, 48), g.normal(70, 48, io="f32"), g.normal(48, io="f32")
    a0, v0, m, s = ssm.layer_norm_fwd(x, w, residual=res, return_stats=True)
    a, v = torch.zeros_like(a0), torch.zeros_like(v0)
    r = ssm.layer_norm_fwd(x, w, residual=res, y=a, residual_out=v)
    assert r[0] is a and r[1] is v and torch.equal(a, a0) and torch.equal(v, v0)
    n0 = ssm.layer_norm_bwd(x, v0, w, m, s, dresidual_out=res)
    ws.fill_(255)
    n1 = ssm.layer_norm_bwd(x, v0, w, m, s, dresidual_out=res, workspace=ws)
    assert all(torch.equal(n0[k], n1[k]) for k in n0)
    n2 = ssm.layer_norm_bwd(x, v0, w, m, s, with_residual=True)   # the stream ends here: no gradient comes in
    n3 = ssm.layer_norm_bwd(x, v0, w, m, s, dresidual_out=torch.zeros_like(res))
    assert n2["dresidual"].dtype == torch.float32 and all(torch.equal(n2[k], n3[k]) for k in n2)
    assert ssm.layer_norm_bwd(x, v0, w, m, s, dresidual_out=res, with_residual=False)["dresidual"] is None


def test_most_rows():
    """The largest batch of a step, one row more, and more rows of a norm than a grid's side takes."""
    import torch
    import selective_state_space_scan_amd as ssm
    B, D, N, W = 65535, 8, 16, 4
    g = Gen(64, "f32")
    x, dl, bm = g.normal(B + 1, D), g.normal(B + 1, D), g.normal(B + 1, N)
    A, w = g.normal(D, N), g.normal(D, W)
    h, cache = g.normal(B + 1, D, N), g.normal(B + 1, W - 1, D)
    sl = torch.randperm(B, generator=g.g).to(DEV, torch.int32)
    h0, c0 = h.clone(), cache.clone()
    y = ssm.selective_scan_step(x[:B], dl[:B], A, bm[:B], bm[:B], None, h, slots=sl)
    yc = ssm.causal_conv_step(x[:B], cache, w, slots=sl)
    at = sl.long()
    hs, cs = h0[at], c0[at]
    half = B // 2
    for part in (slice(0, half), slice(half, B)):
        hp, cp = hs[part].clone(), cs[part].clone()
        assert torch.equal(y[part], ssm.selective_scan_step(x[:B][part], dl[:B][part], A, bm[:B][part], bm[:B][part], None, hp))
        assert torch.equal(yc[part], ssm.causal_conv_step(x[:B][part], cp, w))
        assert torch.equal(h[at[part]], hp) and torch.equal(cache[at[part]], cp)
    for f in (lambda: ssm.selective_scan_step(x, dl, A, bm, bm, None, h), lambda: ssm.causal_conv_step(x, cache, w)):
        with pytest.raises(ssm.SsmScanError) as e:
            f()
        assert e.value.code == ssm.SSM_ERR_UNSUPPORTED
    rows = (1 << 23) + 5
    v, nw = torch.randn((rows, 4), device=DEV), torch.ones(4, device=DEV)
    y, _, m, r = ssm.layer_norm_fwd(v, nw, return_stats=True)
    for part in (slice(0, 50), slice((1 << 23) - 9, rows)):
        yp, _, mp, rp = ssm.layer_norm_fwd(v[part], nw, return_stats=True)
        assert torch.equal(y[part], yp) and torch.equal(m[part], mp) and torch.equal(r[part], rp)
    g = ssm.layer_norm_bwd(y, v, nw, m, r)
    gp = ssm.layer_norm_bwd(y[-40:], v[-40:], nw, m[-40:], r[-40:])
    assert torch.equal(g["dx"][-40:], gp["dx"])


def test_outputs_that_do_not_fit_are_torch_s_out_of_memory():
    """As where torch allocates itself (and in the scan's calls): one exception type to catch, and the next call runs."""
    import torch
    import selective_state_space_scan_amd as ssm
    x, w = torch.ones((1, 1, 1024), dtype=torch.bfloat16, device=DEV), torch.ones((1024, 4), device=DEV)
    big = x.expand(1 << 10, 1 << 20, 1024)   # 2 TiB of output
    for f in (lambda: ssm.causal_conv_fwd(big, w), lambda: ssm.causal_conv_bwd(big, w, None, None, big)):
        with pytest.raises(torch.OutOfMemoryError):
            f()
    y, _ = ssm.causal_conv_fwd(x, w, silu=False)
    assert (y == 1).all()


def test_written_tensors_count_as_modified():
    """torch's version counters see what a call writes, so a graph that saved such a tensor refuses its backward;
    inputs, and tensors without a counter, are left alone."""
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(65, "f32")
    B, L, D, N, W = 2, 9, 16, 16, 4
    x, x3, bm = g.normal(B, D), g.normal(B, L, D), g.normal(B, N)
    A, w, nw = g.normal(D, N), g.normal(D, W), g.normal(D)
    h, h2, c, c2 = g.normal(B, D, N), g.normal(B, D, N), g.normal(B, W - 1, D), g.normal(B, W - 1, D)
    y, y3, y4, c3, r = (torch.zeros_like(t) for t in (x, x3, x3, c, x3))
    ins = [x, x3, bm, A, w, nw]

    def bumped(f, *outs, kept=()):
        old, still = [t._version for t in outs], [t._version for t in (*ins, *kept)]
        f()
        assert all(t._version > v for t, v in zip(outs, old))
        assert [t._version for t in (*ins, *kept)] == still

    bumped(lambda: ssm.selective_scan_step(x, x, A, bm, bm, None, h, y=y), h, y)
    bumped(lambda: ssm.selective_scan_step(x, x, A, bm, bm, None, h, h_last=h2), h2, kept=(h,))
    bumped(lambda: ssm.causal_conv_step(x, c, w, y=y), c, y)
    bumped(lambda: ssm.causal_conv_step(x, c, w, conv_last=c2), c2, kept=(c,))
    bumped(lambda: ssm.causal_conv_fwd(x3, w, y=y3, conv_last=c3), y3, c3)
    bumped(lambda: ssm.causal_conv_bwd(x3, w, None, None, y3, dx=y4), y4, kept=(y3,))
    bumped(lambda: ssm.layer_norm_fwd(x3, nw, y=y3, residual=r, residual_out=r), y3, r)
    bumped(lambda: ssm.layer_norm_fwd(x3, nw, residual=r), kept=(r,))
    p = torch.ones_like(h, requires_grad=True)
    loss = (p * h).sum()   # saves h
    ssm.selective_scan_step(x, x, A, bm, bm, None, h)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    with torch.inference_mode():
        hi = torch.zeros_like(h)
        ssm.selective_scan_step(x, x, A, bm, bm, None, hi)
    assert ssm.selective_scan_step(x, x, A, bm, bm, None, hi).shape == (B, D)


def test_refusals():
    import torch
    import selective_state_space_scan_amd as ssm
    g = Gen(71, "bf16")
    D, W, N = 16, 4, 16
    x, w = g.normal(2, 8, D), g.normal(D, W, io="f32")
    t, bm, A, h = g.normal(2, D), g.normal(2, N), g.normal(D, N, io="f32"), g.normal(2, D, N, io="f32")
    c = g.normal(2, W - 1, D)
    nw = g.normal(D, io="f32")
    bad = [
        lambda: ssm.causal_conv_fwd(x.half(), w), lambda: ssm.causal_conv_fwd(x[0], w),
        lambda: ssm.causal_conv_fwd(x.transpose(1, 2), w), lambda: ssm.causal_conv_fwd(x, w.bfloat16()),
        lambda: ssm.causal_conv_fwd(x, w[:8]), lambda: ssm.causal_conv_fwd(x, w, w[0]),
        lambda: ssm.causal_conv_fwd(x, w, None, torch.zeros(2, device=DEV)),
        lambda: ssm.causal_conv_fwd(x, w, None, torch.zeros(2, dtype=torch.int32)),
        lambda: ssm.causal_conv_fwd(x, w, conv0=c.float()), lambda: ssm.causal_conv_fwd(x, w, conv0=c[:, :2]),
        lambda: ssm.causal_conv_bwd(x, w, None, None, x.float()),
        lambda: ssm.causal_conv_bwd(x, w, None, None, x[..., :1].expand(2, 8, D)),
        lambda: ssm.causal_conv_bwd(x, w, None, None, x, workspace=torch.empty(4, dtype=torch.uint8, device=DEV)),
        lambda: ssm.causal_conv_step(t, c[:1], w), lambda: ssm.causal_conv_step(t, c.transpose(1, 2), w),
        lambda: ssm.causal_conv_step(t, c, w, slots=torch.zeros(2, dtype=torch.int64, device=DEV)),
        lambda: ssm.causal_conv_step(t, c, w, slots=torch.zeros(3, dtype=torch.int32, device=DEV)),
        lambda: ssm.causal_conv_step(x, c, w),
        lambda: ssm.selective_scan_step(t, t, A, bm, bm, None, h.bfloat16()),
        lambda: ssm.selective_scan_step(t, t, A, bm, bm[:, :8], None, h),
        lambda: ssm.selective_scan_step(t, t.float(), A, bm, bm, None, h),
        lambda: ssm.selective_scan_step(t, t, A.t(), bm, bm, None, h[:, :, :8]),
        lambda: ssm.selective_scan_step(t, t, A, bm, bm, None, h, z=x), lambda: ssm.layer_norm_fwd(x.half(), nw),
        lambda: ssm.layer_norm_fwd(x[..., :8], nw[:8]), lambda: ssm.layer_norm_fwd(x, nw[:8]),
        lambda: ssm.layer_norm_fwd(x.float(), nw, residual=x), lambda: ssm.layer_norm_fwd(t, nw, None, i32([1, 1])),
        lambda: ssm.layer_norm_bwd(x.float(), x, nw, None, torch.zeros((2, 8), device=DEV)),
        lambda: ssm.layer_norm_bwd(x, x, nw, None, torch.zeros(16, device=DEV)),
    ]
    for k in (1.5, "x", None):
        bad.append(lambda k=k: ssm.causal_conv_fwd(k, w))
    bad.append(lambda: ssm.selective_scan_step(t, t, A, bm, bm, None, h, delta_clamp=(0.1,)))
    bad.append(lambda: ssm.selective_scan_step(t, t, A, bm, bm, None, h, delta_clamp=0.1))
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            raise AssertionError(i)
    for f, code in ((lambda: ssm.causal_conv_fwd(x, g.normal(D, 5, io="f32")), ssm.SSM_ERR_UNSUPPORTED),
                    (lambda: ssm.causal_conv_fwd(x, w, y=x), ssm.SSM_ERR_ALIAS),
                    (lambda: ssm.causal_conv_fwd(x, w, y=x[:1, :1].expand(2, 8, D)), ssm.SSM_ERR_INVALID_ARG),
                    (lambda: ssm.selective_scan_step(t, t, A, bm, bm, None, h, y=t), ssm.SSM_ERR_ALIAS),
                    (lambda: ssm.selective_scan_step(t, t, A, bm, bm, None, h, delta_clamp=(0.5, 0.1)),
                     ssm.SSM_ERR_INVALID_ARG),
                    (lambda: ssm.layer_norm_fwd(x, nw, eps=0.0), ssm.SSM_ERR_INVALID_ARG),
                    (lambda: ssm.layer_norm_fwd(g.normal(1, 16400), g.normal(16400, io="f32")),
                     ssm.SSM_ERR_UNSUPPORTED)):
        with pytest.raises(ssm.SsmScanError) as e:
            f()
        assert e.value.code == code


# ---- together ------------------------------------------------------------------

class Block:
    """norm -> in-projection -> convolution + silu -> projections -> scan with gate -> out-projection, the block that
    the operators serve, with its forward, its backward and its step on caches, matrix products in float32."""

    def __init__(self, seed, d_model=32, dim=64, N=16, W=4, rank=8):
        import torch
        g = Gen(seed, "f32")
        self.dims = (d_model, dim, N, W, rank)
        self.p = dict(nw=g.normal(d_model, scale=0.1, shift=1.0), nb=g.normal(d_model, scale=0.1),
                      win=g.normal(2 * dim, d_model, scale=d_model ** -0.5), cw=g.normal(dim, W, scale=0.5),
                      cb=g.normal(dim, scale=0.1), wx=g.normal(rank + 2 * N, dim, scale=dim ** -0.5),
                      wd=g.normal(dim, rank, scale=rank ** -0.5),
                      A=torch.log(torch.arange(1, N + 1, device=DEV).float()).repeat(dim, 1), D=g.normal(dim),
                      db=g.normal(dim, scale=0.5, shift=-1.0), wo=g.normal(d_model, dim, scale=dim ** -0.5))

    def forward(self, x, residual, valid_len, save=False):
        import selective_state_space_scan_amd as ssm
        p, (dm, dim, N, W, rank) = self.p, self.dims
        h, v, m, r = ssm.layer_norm_fwd(x, p["nw"], p["nb"], valid_len, residual=residual, return_stats=True)
        xz = h @ p["win"].t()
        xc, conv = ssm.causal_conv_fwd(xz[..., :dim], p["cw"], p["cb"], valid_len)
        q = xc @ p["wx"].t()
        delta = q[..., :rank] @ p["wd"].t()
        Bm, Cm, z = q[..., rank:rank + N].contiguous(), q[..., rank + N:].contiguous(), xz[..., dim:].contiguous()
        kw = dict(delta_bias=p["db"], z=z)
        if save:
            y, state, cs = ssm.selective_scan_fwd(xc, delta, p["A"], Bm, Cm, p["D"], valid_len, **kw,
                                                  return_chunk_states=True, chunk_len=ssm.bwd_chunk_len(N))
            self.saved = (h, v, m, r, xz, xc, q, delta, Bm, Cm, z, cs, y)
        else:
            y, state = ssm.selective_scan_fwd(xc, delta, p["A"], Bm, Cm, p["D"], valid_len, **kw)
        return y @ p["wo"].t(), v, conv, state

    def backward(self, dout, dv, valid_len):
        import torch
        import selective_state_space_scan_amd as ssm
        p, (dm, dim, N, W, rank) = self.p, self.dims
        h, v, m, r, xz, xc, q, delta, Bm, Cm, z, cs, y = self.saved
        two = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        g = dict(wo=two(dout).t() @ two(y))
        s = ssm.selective_scan_bwd(xc, delta, p["A"], Bm, Cm, p["D"], valid_len, dout @ p["wo"], cs,
                                   delta_bias=p["db"], z=z)
        g.update(A=s["dA_log"], D=s["dD"], db=s["ddelta_bias"], wd=two(s["ddelta"]).t() @ two(q[..., :rank]))
        dq = torch.cat([s["ddelta"] @ p["wd"], s["dB"], s["dC"]], -1)
        g["wx"] = two(dq).t() @ two(xc)
        dxz = torch.empty_like(xz)
        dxz[..., dim:] = s["dz"]
        c = ssm.causal_conv_bwd(xz[..., :dim], p["cw"], p["cb"], valid_len, s["dx"] + dq @ p["wx"], dx=dxz[..., :dim])
        g.update(cw=c["dweight"], cb=c["dbias"], win=two(dxz).t() @ two(h))
        n = ssm.layer_norm_bwd(dxz @ p["win"], v, p["nw"], m, r, valid_len, dresidual_out=dv)
        g.update(nw=n["dweight"], nb=n["dbias"], x=n["dx"])
        return g

    def step(self, x, residual, conv, state, slots):
        import selective_state_space_scan_amd as ssm
        p, (dm, dim, N, W, rank) = self.p, self.dims
        h, v = ssm.layer_norm_fwd(x, p["nw"], p["nb"], residual=residual)
        xz = h @ p["win"].t()
        xc = ssm.causal_conv_step(xz[:, :dim], conv, p["cw"], p["cb"], slots=slots)
        q = xc @ p["wx"].t()
        y = ssm.selective_scan_step(xc, q[:, :rank] @ p["wd"].t(), p["A"], q[:, rank:rank + N], q[:, rank + N:],
                                    p["D"], state, delta_bias=p["db"], z=xz[:, dim:], slots=slots)
        return y @ p["wo"].t(), v


def _block_in_64_bits(p, dims, x, residual, lens):
    """The same block from elementary torch operations in float64 on the CPU, row by row; (out, v) with zeros past a
    row's end."""
    import torch
    dm, dim, N, W, rank = dims
    outs, vs = [], []
    for b, n in enumerate(lens):
        v = x[b, :n] + residual[b, :n]
        c = v - v.mean(1, keepdim=True)
        h = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["nw"] + p["nb"]
        xz = h @ p["win"].t()
        xs = torch.cat([torch.zeros((W - 1, dim), dtype=v.dtype), xz[:, :dim]])
        u = p["cb"] + sum(xs[k:k + n] * p["cw"][:, k] for k in range(W))
        u = u * torch.sigmoid(u)
        q = u @ p["wx"].t()
        dt = torch.nn.functional.softplus(q[:, :rank] @ p["wd"].t() + p["db"])
        state, ys = torch.zeros((dim, N), dtype=v.dtype), []
        for t in range(n):
            state = torch.exp(-dt[t][:, None] * torch.exp(p["A"])) * state + (dt[t] * u[t])[:, None] * q[t, rank:rank + N]
            ys.append(state @ q[t, rank + N:] + p["D"] * u[t])
        y = torch.stack(ys) * xz[:, dim:] * torch.sigmoid(xz[:, dim:])
        outs.append(torch.cat([y @ p["wo"].t(), torch.zeros((x.shape[1] - n, dm), dtype=v.dtype)]))
        vs.append(torch.cat([v, torch.zeros((x.shape[1] - n, dm), dtype=v.dtype)]))
    return torch.stack(outs), torch.stack(vs)


def _near(name, got, ref):
    """Chained fp32 operators against 64 bits: the framework's fp32 bar, 1e-4 of the tensor's scale."""
    err = float(np.max(np.abs(n64(got) - ref)) / max(1e-30, np.sqrt(np.mean(ref * ref))))
    assert err <= 1e-3 and float(np.linalg.norm(n64(got) - ref) / np.linalg.norm(ref)) <= 1e-4, (name, err)


def test_block_trains():
    """The operators in the order of a block's forward and backward, all gradients against automatic differentiation
    of the block in 64 bits."""
    import torch
    blk = Block(81)
    g = Gen(82, "f32")
    B, L, dm = 3, 45, 32
    lens = [45, 18, 1]
    x, res, dout, dv = (g.normal(B, L, dm) for _ in range(4))
    for b, n in enumerate(lens):
        dout[b, n:] = 0
        dv[b, n:] = 0
    out, v, _, _ = blk.forward(x, res, i32(lens), save=True)
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
    blk = Block(83)
    dm, dim, N, W, rank = blk.dims
    g = Gen(84, "f32")
    B, prompt, new = 4, 30, 6
    lens = [30, 2, 17, 1]
    x, res = g.normal(B, prompt + new, dm), g.normal(B, prompt + new, dm)
    out0, _, conv, state = blk.forward(x[:, :prompt].contiguous(), res[:, :prompt].contiguous(), i32(lens))
    slots = [5, 0, 7, 3]
    convs, states = torch.full((9, W - 1, dim), 3.0, device=DEV), torch.full((9, dim, N), 3.0, device=DEV)
    convs[slots], states[slots] = conv, state
    # the sequences as they would run in one go: each prompt, then its tokens
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
        want = torch.stack([whole[b, n + t] for b, n in enumerate(lens)])
        _near(f"token {t}", out[:B], n64(want))
        assert (out[B] == 0).all()
    _near("conv", convs[slots], n64(conv_end))
    _near("state", states[slots], n64(state_end))
    rest = [1, 2, 4, 6, 8]
    assert (convs[rest] == 3).all() and (states[rest] == 3).all()
