"""The gated recurrence and the group norm in 64 bits on the CPU, written plainly
from their formulas, each with the largest error that the kernels' fp32
arithmetic may make (U = 2^-24, half a step of fp32; outputs in bf16 add half a
step of bf16).

sigmoid(v) is exp2, an addition and a reciprocal, 2 U, 1 U and 2 U relative, and
for bf16 inputs the rounded exponent: |v| U of e^-v, and 0.25 |v| U for log2(e)'s
own rounding.  exp, exp2, sqrt and rcp count 2 U each (1 ulp)."""
from __future__ import annotations

import numpy as np

from block_ref import U, lengths, out_step, sigmoid


def sig_err(v, io):
    """Relative error of sigmoid(v)."""
    return (6 + (1.25 if io == "bf16" else 0) * np.abs(v)) * U


# ---- gated recurrence --------------------------------------------------------

def _gates(ag, xg, A_log, io):
    """r, i, s, a, c and the relative errors of r, i, s, a, c."""
    r, i = sigmoid(ag), sigmoid(xg)
    s = np.exp(A_log) * r
    a = np.exp(-s)
    c2 = -np.expm1(-2 * s)
    c = np.sqrt(c2)
    er, ei = sig_err(ag, io), sig_err(xg, io)
    # exp(A_log) 2 U, its products with log2(e), r and ln 2, and the constants' own rounding
    es = er + 7 * U
    ea = s * es + 3 * U
    # the polynomial: its argument's error (condition at most 1), its steps and its distance; the difference: a^2's error
    near = es + 9 * U
    with np.errstate(divide="ignore", invalid="ignore"):
        far = np.where(c2 > 0, 2 * a * a / c2 * ea, 0) + 2 * U
    ec = 0.5 * np.where(2 * s < 0.49, near, np.maximum(near, far)) + 2 * U
    return r, i, s, a, c, er, ei, es, ea, ec


def gated_fwd(x, ag, xg, A_log, valid_len=None, h0=None, io="f32", chunk=64):
    """(y, h_last, chunk_states) and their tolerances.

    A state's error: what the one in front brings, a's own error and the roundings of products of decays and of the
    sums that compose them, each on the sum of magnitudes (m) that reaches the step."""
    B, L, D = x.shape
    nc = -(-L // chunk)
    y, ye = np.zeros((B, L, D)), np.zeros((B, L, D))
    last, le = np.zeros((B, D)), np.zeros((B, D))
    st, se = np.zeros((B, nc, D)), np.zeros((B, nc, D))
    for b, n in enumerate(lengths(valid_len, B, L)):
        r, i, s, a, c, er, ei, es, ea, ec = _gates(ag[b, :n], xg[b, :n], A_log, io)
        u = c * i * x[b, :n]
        eu = np.abs(u) * (ec + ei + 3 * U)
        h = np.zeros(D) if h0 is None else h0[b].astype(np.float64)
        m, he = np.abs(h), np.zeros(D)
        for t in range(L):
            if t < n:
                he = a[t] * he + a[t] * m * (ea[t] + 3 * U) + eu[t]
                h, m = a[t] * h + u[t], a[t] * m + np.abs(u[t])
                he = he + 3 * U * m
                y[b, t], ye[b, t] = h, he
            if t % chunk == chunk - 1 or t == L - 1:
                st[b, t // chunk], se[b, t // chunk] = h, he
        last[b], le[b] = h, he
    return (y, last, st), (ye + out_step(io) * np.abs(y) * 1.01, le, se)


def gated_bwd(x, ag, xg, A_log, valid_len, dy, h0=None, dh_last=None, io="f32"):
    """Gradients and their tolerances, two dicts: dx, da_gate, dx_gate, dA_log, dh0."""
    B, L, D = x.shape
    z = lambda *s: np.zeros(s)  # noqa: E731
    out = dict(dx=z(B, L, D), da_gate=z(B, L, D), dx_gate=z(B, L, D), dA_log=z(D), dh0=z(B, D))
    tol = {k: np.zeros_like(v) for k, v in out.items()}
    mag = np.zeros(D)
    for b, n in enumerate(lengths(valid_len, B, L)):
        r, i, s, a, c, er, ei, es, ea, ec = _gates(ag[b, :n], xg[b, :n], A_log, io)
        xb = x[b, :n].astype(np.float64)
        u = c * i * xb
        eu = np.abs(u) * (ec + ei + 3 * U)
        h = np.zeros(D) if h0 is None else h0[b].astype(np.float64)
        m, he = np.abs(h), U * np.abs(h)
        hp, hpe = np.zeros((n, D)), np.zeros((n, D))
        for t in range(n):
            hp[t], hpe[t] = h, he
            he = a[t] * he + a[t] * m * (ea[t] + 3 * U) + eu[t]
            h, m = a[t] * h + u[t], a[t] * m + np.abs(u[t])
            he = he + 3 * U * m
        g = np.zeros(D) if dh_last is None else dh_last[b].astype(np.float64)
        gm, ge = np.abs(g), np.zeros(D)
        for t in range(n - 1, -1, -1):
            G, Ge = g + dy[b, t], ge + 3 * U * (gm + np.abs(dy[b, t]))
            Gm = gm + np.abs(dy[b, t])
            out["dx"][b, t] = G * i[t] * c[t]
            tol["dx"][b, t] = np.abs(G * i[t] * c[t]) * (ei[t] + ec[t] + 3 * U) + Ge * i[t] * c[t]
            gxc = G * i[t] * xb[t] * c[t]
            out["dx_gate"][b, t] = gxc * (1 - i[t])
            tol["dx_gate"][b, t] = (np.abs(gxc) * ((1 - i[t]) * (ei[t] + ec[t] + 5 * U) + i[t] * ei[t] + U)
                                    + Ge * np.abs(i[t] * xb[t] * c[t] * (1 - i[t])))
            sa = s[t] * a[t]
            with np.errstate(divide="ignore", invalid="ignore"):
                ratio = np.where(c[t] > 0, sa * a[t] / c[t], 0.0)
            p1, p2 = ratio * G * i[t] * xb[t], sa * G * hp[t]
            q = p1 - p2
            qe = (np.abs(p1) * (es[t] + 2 * ea[t] + ec[t] + ei[t] + 9 * U) + np.abs(ratio * i[t] * xb[t]) * Ge
                  + np.abs(p2) * (es[t] + ea[t] + 4 * U) + sa * (np.abs(hp[t]) * Ge + np.abs(G) * hpe[t])
                  + U * (np.abs(p1) + np.abs(p2)))
            out["da_gate"][b, t] = q * (1 - r[t])
            tol["da_gate"][b, t] = qe * (1 - r[t]) + np.abs(q) * (r[t] * er[t] + 2 * U)
            out["dA_log"] += q
            tol["dA_log"] += qe
            mag += np.abs(q)
            ge = a[t] * Ge + a[t] * Gm * (ea[t] + 3 * U)
            g, gm = a[t] * G, a[t] * Gm
        out["dh0"][b], tol["dh0"][b] = g, ge + 2 * U * gm
    # a lane adds every eighth step of a row at most, then the waves, tiles and rows join
    tol["dA_log"] += (L / 8 + 100) * U * mag
    for k in ("dx", "da_gate", "dx_gate"):
        tol[k] += out_step(io) * np.abs(out[k]) * 1.01
    return out, tol


# ---- group norm --------------------------------------------------------------

def _act(u, silu):
    """act(u), act'(u)."""
    if not silu:
        return u, np.ones_like(u)
    s = sigmoid(u)
    return u * s, s * (1 + u * (1 - s))


def _act_err(u, silu, io):
    """Errors of act(u) relative and of act'(u) absolute, u exact."""
    if not silu:
        return np.zeros_like(u), np.zeros_like(u)
    return sig_err(u, io) + 2 * U, 16 * U * (1 + np.abs(u)) + np.abs(u) * sig_err(u, io)


def group_fwd(x, groups, w, bias, z=None, silu=True, gate_first=False, eps=1e-5, rms=False, io="f32", depth=48):
    """(y, mean, rstd) and their tolerances for rows [rows, dim].
    depth: additions behind one another in a group's sum."""
    R, D = x.shape
    shape = (R, groups, D // groups)
    v, ve = x.astype(np.float64), np.zeros((R, D))
    if z is not None and gate_first:
        act, _ = _act(z, silu)
        v = v * act
        ve = np.abs(v) * (_act_err(z, silu, io)[0] + U)
    v, ve = v.reshape(shape), ve.reshape(shape)
    m = np.zeros(shape[:2]) if rms else v.mean(2)
    cc = v - m[..., None]
    ce = ve + 2 * U * np.abs(cc)
    me = np.zeros_like(m)
    if not rms:
        # the rounded mean is corrected by the sum of differences from it: what remains is that sum's own error
        me = ve.mean(2) + depth * U * (np.abs(cc).mean(2) + U * depth * np.abs(v).mean(2))
        ce = ce + me[..., None]
    var = (cc * cc).mean(2)
    r = 1 / np.sqrt(var + eps)
    rel = depth * U + 2 * (np.abs(cc) * ce).mean(2) / (var + eps)
    re = r * (0.5 * rel + 6 * U)
    xh = (cc * r[..., None]).reshape(R, D)
    xe = (ce * r[..., None] + np.abs(cc) * re[..., None]).reshape(R, D) + 2 * U * np.abs(xh)
    p = xh * w + (0 if bias is None else bias)
    pe = np.abs(w) * xe + U * np.abs(xh * w) + U * np.abs(p)
    if z is None:
        y = _act(p, silu)[0]
        ye = (1.1 if silu else 1) * pe + np.abs(y) * _act_err(p, silu, io)[0]
    elif gate_first:
        y, ye = p, pe
    else:
        act = _act(z, silu)[0]
        y = p * act
        ye = pe * np.abs(act) + np.abs(y) * (_act_err(z, silu, io)[0] + U)
    return (y, m, r), (ye + out_step(io) * np.abs(y) * 1.01, me + 2 * U * np.abs(m), re)


def group_bwd(dy, x, groups, w, bias, mean, rstd, z=None, silu=True, gate_first=False, io="f32", depth=48,
              rows_depth=128):
    """Gradients and tolerances for rows [rows, dim], two dicts: dx, dz, dweight, dbias."""
    R, D = x.shape
    shape = (R, groups, D // groups)
    x = x.astype(np.float64)
    v, ve = x, np.zeros((R, D))
    if z is not None and gate_first:
        v = x * _act(z, silu)[0]
        ve = np.abs(v) * (_act_err(z, silu, io)[0] + U)
    each = lambda t: np.repeat(t, D // groups, axis=1)  # noqa: E731  one value a group, for its channels
    r = each(rstd.astype(np.float64))
    xh = (v - (0 if mean is None else each(mean))) * r
    xe = 3 * U * np.abs(xh) + ve * r
    p = xh * w + (0 if bias is None else bias)
    pe = np.abs(w) * xe + U * np.abs(xh * w) + U * np.abs(p)
    dz = dze = None
    dp, dpe = dy.astype(np.float64), np.zeros((R, D))
    if z is None:
        slope = _act(p, silu)[1]
        dpe = np.abs(dp) * ((0.5 * pe if silu else 0) + _act_err(p, silu, io)[1] + U * np.abs(slope))
        dp = dp * slope
    elif not gate_first:
        act, slope = _act(z, silu)
        ae, se = _act_err(z, silu, io)
        dz = dp * p * slope
        dze = np.abs(dp) * (pe * np.abs(slope) + np.abs(p) * se) + 2 * U * np.abs(dz)
        dpe = np.abs(dp * act) * (ae + U)
        dp = dp * act
    k = dp * w
    ke = np.abs(w) * dpe + U * np.abs(k)
    over = lambda t: each(t.reshape(shape).mean(2))  # noqa: E731
    along, ale = over(k * xh), over(depth * U * np.abs(k * xh) + np.abs(k) * xe + ke * np.abs(xh))
    inner = k - xh * along
    ie = ke + 2 * U * np.abs(k) + xe * np.abs(along) + np.abs(xh) * ale + 3 * U * np.abs(xh * along)
    if mean is not None:
        inner = inner - over(k)
        ie = ie + over(ke + depth * U * np.abs(k)) + 2 * U * np.abs(inner)
    dv = inner * r
    de = (ie + 2 * U * np.abs(inner)) * r
    dx, dxe = dv, de
    if z is not None and gate_first:
        act, slope = _act(z, silu)
        ae, se = _act_err(z, silu, io)
        dz = dv * x * slope
        dze = de * np.abs(x * slope) + np.abs(dv * x) * se + 3 * U * np.abs(dz)
        dx = dv * act
        dxe = de * np.abs(act) + np.abs(dx) * (ae + U)
    out = dict(dx=dx, dz=dz, dweight=(dp * xh).sum(0), dbias=None if bias is None else dp.sum(0))
    tol = dict(dx=dxe + out_step(io) * np.abs(dx) * 1.01,
               dz=None if dz is None else dze + out_step(io) * np.abs(dz) * 1.01,
               dweight=(np.abs(dp) * (xe + rows_depth * U * np.abs(xh)) + dpe * np.abs(xh)).sum(0),
               dbias=None if bias is None else (dpe + rows_depth * U * np.abs(dp)).sum(0))
    return out, tol
