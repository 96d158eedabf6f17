"""The operators beside the scan (short causal convolution, single-token steps,
norms) in 64 bits on the CPU, written plainly from their formulas, each with the
largest error that the kernels' fp32 arithmetic may make.

A tolerance counts roundings: U = 2^-24 is half a step of fp32.  An output
stored in bf16 adds half a step of bf16, 2^-8 of its value.  Sums count one
rounding of the running value per addition of a lane's own chain and of the tree
that joins the lanes (the depths below), each bounded by the sum of magnitudes.
sigmoid, softplus and exp2 are good to a few U relative to their value; the
counts allow for 1 ulp (2 U) of v_exp_f32, v_log_f32 and v_rcp_f32 each and
their surrounding multiplications."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def out_step(io: str) -> float:
    return 2.0 ** -8 if io == "bf16" else U


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def lengths(valid_len, B, L):
    return [L] * B if valid_len is None else [int(min(max(n, 0), L)) for n in valid_len]


# ---- convolution -------------------------------------------------------------

def conv_fwd(x, w, bias, valid_len=None, conv0=None, silu=True, io="f32"):
    """y, conv_last and y's tolerance."""
    B, L, D = x.shape
    W = w.shape[1]
    y, tol = np.zeros((B, L, D)), np.zeros((B, L, D))
    last = np.zeros((B, W - 1, D))
    for b, n in enumerate(lengths(valid_len, B, L)):
        xs = np.zeros((W - 1 + n, D))
        if conv0 is not None:
            xs[:W - 1] = conv0[b]
        xs[W - 1:] = x[b, :n]
        for t in range(n):
            p = np.zeros(D) if bias is None else bias.astype(np.float64).copy()
            mag = np.abs(p)
            for k in range(W):
                p = p + w[:, k] * xs[t + k]
                mag = mag + np.abs(w[:, k] * xs[t + k])
            y[b, t] = p * sigmoid(p) if silu else p
            # W products and sums on values up to mag; |silu'| <= 1.1; 10 U for the sigmoid and its product
            tol[b, t] = 1.1 * (W + 1) * U * mag + 10 * U * np.abs(y[b, t])
        last[b] = xs[n:]
    return y, last, tol + out_step(io) * np.abs(y) * 1.01


def conv_bwd(x, w, bias, valid_len, dy, conv0=None, dconv_last=None, silu=True, io="f32", depth=128):
    """Gradients and their tolerances, two dicts: dx, dweight, dbias, dconv0.
    depth: additions behind one another in a weight gradient's sum."""
    B, L, D = x.shape
    W = w.shape[1]
    z = lambda *s: np.zeros(s)  # noqa: E731
    out = dict(dx=z(B, L, D), dweight=z(D, W), dbias=z(D), dconv0=z(B, W - 1, D))
    tol = {k: np.zeros_like(v) for k, v in out.items()}
    for b, n in enumerate(lengths(valid_len, B, L)):
        xs = np.zeros((W - 1 + n, D))
        if conv0 is not None:
            xs[:W - 1] = conv0[b]
        xs[W - 1:] = x[b, :n]
        g, ge = np.zeros((n, D)), np.zeros((n, D))
        for t in range(n):
            p = np.zeros(D) if bias is None else bias.astype(np.float64).copy()
            mag = np.abs(p)
            for k in range(W):
                p = p + w[:, k] * xs[t + k]
                mag = mag + np.abs(w[:, k] * xs[t + k])
            if silu:
                s = sigmoid(p)
                g[t] = dy[b, t] * s * (1 + p * (1 - s))
                # |d silu'/dp| <= 0.5 on p's error; 1 - s, the product and the sum: 16 U of (1 + |p|)
                ge[t] = np.abs(dy[b, t]) * U * (0.5 * (W + 1) * mag + 16 * (1 + np.abs(p)))
            else:
                g[t] = dy[b, t]
        dxs, dxe = np.zeros((W - 1 + n, D)), np.zeros((W - 1 + n, D))
        for t in range(n):
            for k in range(W):
                dxs[t + k] += w[:, k] * g[t]
                dxe[t + k] += np.abs(w[:, k]) * (ge[t] + (W + 2) * U * np.abs(g[t]))
                out["dweight"][:, k] += g[t] * xs[t + k]
                tol["dweight"][:, k] += np.abs(xs[t + k]) * (ge[t] + depth * U * np.abs(g[t]))
            out["dbias"] += g[t]
            tol["dbias"] += ge[t] + depth * U * np.abs(g[t])
        if dconv_last is not None:
            dxs[n:] += dconv_last[b]
            dxe[n:] += U * np.abs(dconv_last[b])
        dxe += U * np.abs(dxs)
        out["dconv0"][b], tol["dconv0"][b] = dxs[:W - 1], dxe[:W - 1]
        out["dx"][b, :n], tol["dx"][b, :n] = dxs[W - 1:], dxe[W - 1:]
    for k in ("dx", "dconv0"):
        tol[k] += out_step(io) * np.abs(out[k]) * 1.01
    for k in ("dweight", "dbias"):
        tol[k] += U * np.abs(out[k])
    return out, tol


# ---- the scan's step ---------------------------------------------------------

def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def scan_step(x, delta, A_log, B, C, D, h, delta_bias=None, z=None, softplus_on=True, clamp=None, io="f32"):
    """y, h' and their tolerances for rows that all take the step (h as the batch's rows)."""
    raw = delta if delta_bias is None else delta + delta_bias
    dt = softplus(raw) if softplus_on else raw
    # the sum with the bias, and softplus to 4 U of its value (its derivative is below its value)
    dte = np.abs(dt) * U * 6 + np.abs(raw) * U * np.minimum(1, np.abs(dt))
    if clamp is not None:
        dt = np.clip(dt, *clamp)
    A = -np.exp(A_log.astype(np.float64))
    ex = dt[..., None] * A
    decay = np.exp(ex)
    # A to (4 + 2 |A_log|) U, its products with log2(e) and delta, and exp2 itself
    dece = decay * (np.abs(ex) * U * (10 + 2 * np.abs(A_log)) + np.abs(A) * dte[..., None] + 3 * U)
    u = (dt * x)[..., None] * B[:, None, :]
    ue = (dte * np.abs(x))[..., None] * np.abs(B[:, None, :]) + 3 * U * np.abs(u)
    new = decay * h + u
    he = np.abs(h) * dece + ue + 2 * U * (np.abs(decay * h) + np.abs(u))
    y = (new * C[:, None, :]).sum(-1)
    N = A_log.shape[1]
    ye = (np.abs(C[:, None, :]) * (he + (N / 4 + 6) * U * np.abs(new))).sum(-1)
    if D is not None:
        y = y + D * x
        ye = ye + 2 * U * (np.abs(D * x) + np.abs(y))
    if z is not None:
        gate = z * sigmoid(z)
        ye = ye * np.abs(gate) + 12 * U * np.abs(y * gate)
        y = y * gate
    return y, new, ye + out_step(io) * np.abs(y) * 1.01, he


# ---- norms -------------------------------------------------------------------

def norm_fwd(x, w, bias, residual=None, eps=1e-5, rms=False, io="f32", rio="f32", depth=48):
    """(y, v, mean, rstd) and their tolerances for rows [rows, dim].
    depth: additions behind one another in a row's sum."""
    v = x.astype(np.float64) if residual is None else x.astype(np.float64) + residual
    ve = np.zeros_like(v) if residual is None else U * np.abs(v)
    m = np.zeros(v.shape[0]) if rms else v.mean(1)
    c = v - m[:, None]
    spread = np.abs(c).mean(1)
    ce = ve + U * np.abs(c) * 2
    me = np.zeros_like(m)
    if not rms:
        # the rounded mean is corrected by the sum of differences from it: what remains is that sum's own error
        me = ve.mean(1) + depth * U * (spread + U * depth * np.abs(v).mean(1))
        ce = ce + me[:, None]
    var = (c * c).mean(1)
    r = 1 / np.sqrt(var + eps)
    # relative error of var: its chain, and the differences' errors
    rel = depth * U + 2 * (np.abs(c) * ce).mean(1) / (var + eps)
    re = r * (0.5 * rel + 6 * U)
    xh = c * r[:, None]
    y = xh * w
    ye = np.abs(w) * (ce * r[:, None] + np.abs(c) * re[:, None] + 3 * U * np.abs(xh))
    if bias is not None:
        y = y + bias
    ye = ye + U * np.abs(y)
    out = (y, v, m, r)
    tol = (ye + out_step(io) * np.abs(y) * 1.01, ve + out_step(rio) * np.abs(v) * 1.01, me + 2 * U * np.abs(m), re)
    return out, tol


def norm_bwd(dy, v, w, mean, rstd, dresidual_out=None, io="f32", rio="f32", depth=48, rows_depth=128):
    """Gradients and tolerances for rows [rows, dim], two dicts: dx, dresidual, dweight, dbias."""
    r = rstd[:, None].astype(np.float64)
    c = v - (0 if mean is None else mean[:, None])
    xh = c * r
    xe = 3 * U * np.abs(xh)
    g = dy * w
    along = (g * xh).mean(1)[:, None]
    along_e = (depth * U * np.abs(g * xh) + np.abs(g) * xe).mean(1)[:, None]
    inner = g - xh * along
    ie = 2 * U * np.abs(g) + xe * np.abs(along) + np.abs(xh) * along_e + 3 * U * np.abs(xh * along)
    if mean is not None:
        inner = inner - g.mean(1)[:, None]
        ie = ie + depth * U * np.abs(g).mean(1)[:, None] + 2 * U * np.abs(inner)
    dv = inner * r
    de = (ie + 2 * U * np.abs(inner)) * r
    if dresidual_out is not None:
        dv = dv + dresidual_out
        de = de + U * np.abs(dv)
    out = dict(dx=dv, dresidual=dv, dweight=(dy * xh).sum(0), dbias=dy.sum(0))
    tol = dict(dx=de + out_step(io) * np.abs(dv) * 1.01, dresidual=de + out_step(rio) * np.abs(dv) * 1.01,
               dweight=(np.abs(dy) * (xe + rows_depth * U * np.abs(xh))).sum(0),
               dbias=(rows_depth * U * np.abs(dy)).sum(0))
    return out, tol


def check(name, got, ref, tol):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if ref.size == 0:
        return
    bad = ~(np.abs(got - ref) <= tol + 1e-37)   # fp32 results below its normal range may be flushed
    if bad.any():
        i = tuple(int(k) for k in np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]!r} for {ref[i]!r}, "
                             f"allowed {tol[i]!r}")
