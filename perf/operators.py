"""The operators around the selective scan: what is measured of them, and their plain forms.

Six directions of four operators, each as the block around the scan uses it:

* ``conv_fwd``, ``conv_bwd``: the short causal convolution over whole sequences (prompts and training);
* ``conv_step``: the same for one token of every sequence, on the cache of its last inputs;
* ``scan_step``: the selective scan for one token of every sequence, on the cache of states;
* ``norm_fwd``, ``norm_bwd``: layer norm or RMS norm with the residual add in front of it.

``run`` computes them from elementary torch operations in 32 bits, or, with ``own``, calls the framework.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # A short float32 prompt: the smallest call, where latency counts.
        dict(name="conv_fwd-f32-b2-l256-d64-w4", op="conv_fwd", io="f32", batch=2, seqlen=256, dim=64, width=4, bias=True,
             silu=True, wide=False, ragged=False, carry=False),
        # Prompts of different lengths, continued from earlier pieces; x is one half of the in-projection's output.
        dict(name="conv_fwd-bf16-b16-l8192-d512-w4", op="conv_fwd", io="bf16", batch=16, seqlen=8192, dim=512, width=4,
             bias=True, silu=True, wide=True, ragged=True, carry=True),
        # An odd float32 training batch without activation, gradients through the carried inputs.
        dict(name="conv_bwd-f32-b3-l1021-d200-w3", op="conv_bwd", io="f32", batch=3, seqlen=1021, dim=200, width=3,
             bias=False, silu=False, wide=False, ragged=True, carry=True),
        # A training step at the scan's headline size.
        dict(name="conv_bwd-bf16-b8-l4096-d1024-w4", op="conv_bwd", io="bf16", batch=8, seqlen=4096, dim=1024, width=4,
             bias=True, silu=True, wide=True, ragged=False, carry=False),
        # One user's next token.
        dict(name="conv_step-bf16-b1-d2048-w4", op="conv_step", io="bf16", batch=1, dim=2048, width=4, bias=True, silu=True,
             slots=0, idle=0),
        # The next token of a full serving batch, its sequences anywhere in a cache that holds twice as many.
        dict(name="conv_step-bf16-b256-d2048-w4", op="conv_step", io="bf16", batch=256, dim=2048, width=4, bias=True,
             silu=True, slots=512, idle=3),
        # One user's next token.
        dict(name="scan_step-bf16-b1-d2048-n16", op="scan_step", io="bf16", batch=1, dim=2048, dstate=16, gate=True,
             skip=True, clamp=False, slots=0, idle=0),
        # The next token of a full serving batch.
        dict(name="scan_step-bf16-b256-d2048-n16", op="scan_step", io="bf16", batch=256, dim=2048, dstate=16, gate=True,
             skip=True, clamp=False, slots=512, idle=3),
        # The norm in front of a block for a handful of sequences' next token, at an odd width.
        dict(name="norm_fwd-f32-r24-d1000", op="norm_fwd", io="f32", rows=24, dim=1000, rms=True, residual="none", bias=False),
        # The same over a training batch at the scan's headline size, residual stream in float32.
        dict(name="norm_fwd-bf16-r32768-d1024", op="norm_fwd", io="bf16", rows=32768, dim=1024, rms=False, residual="f32",
             bias=True),
        # An odd float32 training batch.
        dict(name="norm_bwd-f32-r1021-d600", op="norm_bwd", io="f32", rows=1021, dim=600, rms=False, residual="none",
             bias=True),
        # A training step at the scan's headline size, residual stream in float32.
        dict(name="norm_bwd-bf16-r32768-d1024", op="norm_bwd", io="bf16", rows=32768, dim=1024, rms=True, residual="f32",
             bias=False),
    ]


MAX_ELEMENTS = 8 * 4096 * 1024   # of one [batch, length, dim] tensor, or of the states


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A width: half of them multiples of 64, as models have them, the others anything."""
    d = _log_uniform(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_step", "norm_fwd", "norm_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("conv_fwd", "conv_bwd"):
        dim = _dim(rng, 16, 2048)
        batch = _log_uniform(rng, 1, 16)
        seqlen = _log_uniform(rng, 1, max(1, min(32768, MAX_ELEMENTS // (dim * batch))))
        return dict(op=op, io=io, batch=batch, seqlen=seqlen, dim=dim, width=rng.choice([2, 3, 4, 4]), bias=flip(),
                    silu=flip(), wide=flip(), ragged=flip(), carry=flip())
    if op in ("conv_step", "scan_step"):
        batch = _log_uniform(rng, 1, 512)
        slots = 2 * batch if flip() else 0
        idle = rng.randint(0, batch // 8) if slots else 0
        if op == "conv_step":
            return dict(op=op, io=io, batch=batch, dim=_dim(rng, 16, 4096), width=rng.choice([2, 3, 4, 4]), bias=flip(),
                        silu=flip(), slots=slots, idle=idle)
        dstate = rng.choice([16, 16, 32, 64])
        dim = _dim(rng, 16, max(16, min(4096, MAX_ELEMENTS // 4 // (batch * dstate))))
        return dict(op=op, io=io, batch=batch, dim=dim, dstate=dstate, gate=flip(), skip=flip(), clamp=flip(),
                    slots=slots, idle=idle)
    dim = _dim(rng, 16, 8192)
    residual = rng.choice(["none", "same", "f32"])
    return dict(op=op, io=io, rows=_log_uniform(rng, 1, MAX_ELEMENTS // dim), dim=dim, rms=flip(),
                residual=residual, bias=flip())


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["io"]]
    dev = "cuda"

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device=dev) * scale + shift).to(dtype)

    def uniform(*shape, bound):
        return (torch.rand(shape, generator=g, device=dev) * 2 - 1) * bound

    s = dict(case=case)
    op, D = case["op"], case["dim"]
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        W = case["width"]
        s["weight"] = uniform(D, W, bound=W ** -0.5)   # a depthwise convolution's usual initial range
        s["bias"] = uniform(D, bound=W ** -0.5) if case["bias"] else None
    if op in ("conv_fwd", "conv_bwd"):
        B, L = case["batch"], case["seqlen"]
        s["x"] = normal(B, L, 2 * D)[..., :D] if case["wide"] else normal(B, L, D)
        s["valid_len"] = (torch.randint(0, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
                          if case["ragged"] else None)
        s["conv0"] = normal(B, W - 1, D) if case["carry"] else None
        if op == "conv_bwd":
            s["dy"] = normal(B, L, D)
            s["dconv_last"] = normal(B, W - 1, D) if case["carry"] else None
    elif op in ("conv_step", "scan_step"):
        B = case["batch"]
        n = case["slots"] or B
        s["slots"] = None
        if case["slots"]:
            slots = torch.randperm(n, generator=g, device=dev)[:B].to(torch.int32)
            if case["idle"]:
                slots[B - case["idle"]:] = -1   # rows that pad the batch
            s["slots"] = slots
        if op == "conv_step":
            s["x"] = normal(B, 2 * D)[:, :D]   # one half of the in-projection's output
            s["conv"] = normal(n, W - 1, D)
            s["conv_last"] = torch.zeros_like(s["conv"])
            s["y"] = torch.empty((B, D), dtype=dt, device=dev)
        else:
            N = case["dstate"]
            s["x"] = normal(B, D)
            s["delta"] = normal(B, D, scale=0.5, shift=-4.0)
            bc = normal(B, 2 * N)   # both come out of one projection
            s["B"], s["C"] = bc[:, :N], bc[:, N:]
            s["z"] = normal(B, 2 * D)[:, D:] if case["gate"] else None
            s["A_log"] = torch.log(torch.arange(1, N + 1, device=dev, dtype=torch.float32)).repeat(D, 1).contiguous()
            s["D"] = normal(D, dtype=torch.float32) if case["skip"] else None
            s["delta_bias"] = normal(D, dtype=torch.float32, scale=0.1)
            s["clamp"] = (1e-3, 0.1) if case["clamp"] else None
            s["h"] = normal(n, D, N, dtype=torch.float32)
            s["h_last"] = torch.zeros_like(s["h"])
            s["y"] = torch.empty((B, D), dtype=dt, device=dev)
    else:
        R = case["rows"]
        rdt = torch.float32 if case["residual"] == "f32" else dt
        s["eps"] = 1e-5
        s["weight"] = normal(D, dtype=torch.float32, scale=0.1, shift=1.0)
        s["bias"] = normal(D, dtype=torch.float32, scale=0.1) if case["bias"] else None
        if op == "norm_fwd":
            s["x"] = normal(R, D)
            s["residual"] = None if case["residual"] == "none" else normal(R, D, dtype=rdt, scale=2.0, shift=0.3)
        else:
            s["v"] = normal(R, D, dtype=rdt, scale=2.0, shift=0.3)   # what the forward normalised
            v = s["v"].double()
            mean = torch.zeros(R, dtype=torch.float64, device=dev) if case["rms"] else v.mean(1)
            s["rstd"] = (((v - mean[:, None]) ** 2).mean(1) + s["eps"]).rsqrt().float()
            s["mean"] = None if case["rms"] else mean.float()
            s["dy"] = normal(R, D)
            s["dresidual_out"] = None if case["residual"] == "none" else normal(R, D, dtype=rdt)
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _conv_inputs(s):
    """The inputs in 32 bits behind the carried ones, [batch, width - 1 + length, dim], zero past a row's end, and which
    steps are valid, [batch, length, 1]."""
    x = s["x"].float()
    B, L, D = x.shape
    W = s["weight"].shape[1]
    t = torch.arange(L, device=x.device)
    n = torch.full((B,), L, device=x.device) if s["valid_len"] is None else s["valid_len"].long().clamp(0, L)
    valid = (t[None, :] < n[:, None])[..., None]
    x = torch.where(valid, x, torch.zeros_like(x))
    front = x.new_zeros((B, W - 1, D)) if s["conv0"] is None else s["conv0"].float()
    return torch.cat([front, x], 1), valid, n


def _conv_last_steps(n, W):
    """Where the last width - 1 inputs of rows of length n stand behind the carried ones."""
    return n[:, None] + torch.arange(W - 1, device=n.device)[None, :]


def _plain_conv_fwd(s):
    xs, valid, n = _conv_inputs(s)
    W, dt, D = s["weight"].shape[1], s["x"].dtype, xs.shape[2]
    p = (xs.unfold(1, W, 1) * s["weight"]).sum(-1)
    if s["bias"] is not None:
        p = p + s["bias"]
    y = p * _sigmoid(p) if s["case"]["silu"] else p
    y = torch.where(valid, y, torch.zeros_like(y)).to(dt)
    last = xs.gather(1, _conv_last_steps(n, W)[..., None].expand(-1, -1, D)).to(dt)
    return {"y": y, "conv_last": last}


def _plain_conv_bwd(s):
    xs, valid, n = _conv_inputs(s)
    w, dt, D = s["weight"], s["x"].dtype, xs.shape[2]
    W, L = w.shape[1], s["x"].shape[1]
    g = s["dy"].float()
    if s["case"]["silu"]:
        p = (xs.unfold(1, W, 1) * w).sum(-1)
        if s["bias"] is not None:
            p = p + s["bias"]
        sg = _sigmoid(p)
        g = g * sg * (1 + p * (1 - sg))
    g = torch.where(valid, g, torch.zeros_like(g))
    dw = (xs.unfold(1, W, 1).double() * g.double()[..., None]).sum((0, 1)).float()
    db = g.double().sum((0, 1)).float() if s["bias"] is not None else None
    # an input reaches the W steps from its own on, the first through the last tap
    edge = g.new_zeros((g.shape[0], W - 1, D))
    dxs = (torch.cat([edge, g, edge], 1).unfold(1, W, 1) * w.flip(1)).sum(-1)
    if s["dconv_last"] is not None:
        at = _conv_last_steps(n, W)[..., None].expand(-1, -1, D)
        dxs = dxs.scatter_add(1, at, s["dconv_last"].float())
    return {"dx": dxs[:, W - 1:].to(dt), "dweight": dw, "dbias": db,
            "dconv0": dxs[:, :W - 1].to(dt) if s["conv0"] is not None else None}


def _pick(s, cache):
    """The rows of a cache that a step's batch reads, and which of the batch are active."""
    if s["slots"] is None:
        return cache, None, None
    active = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    return cache[at], active, at


def _put(s, out, new, active, at):
    if s["slots"] is None:
        out.copy_(new)
    else:
        # the idle rows write a spare row behind the cache
        ext = torch.cat([out, out[:1]])
        ext[torch.where(active, at, torch.full_like(at, out.shape[0]))] = new.to(out.dtype)
        out.copy_(ext[:-1])
    return out


def _plain_conv_step(s):
    conv, active, at = _pick(s, s["conv"])
    xs = torch.cat([conv, s["x"][:, None]], 1)
    p = (xs.float() * s["weight"].t()[None]).sum(1)
    if s["bias"] is not None:
        p = p + s["bias"]
    y = p * _sigmoid(p) if s["case"]["silu"] else p
    if active is not None:
        y = torch.where(active[:, None], y, torch.zeros_like(y))
    return {"y": y.to(s["x"].dtype), "conv_last": _put(s, s["conv_last"], xs[:, 1:], active, at)}


def _plain_scan_step(s):
    h, active, at = _pick(s, s["h"])
    x = s["x"].float()
    delta = _softplus(s["delta"].float() + s["delta_bias"])
    if s["clamp"] is not None:
        delta = torch.clamp(delta, s["clamp"][0], s["clamp"][1])
    decay = torch.exp(-torch.exp(s["A_log"])[None] * delta[..., None])
    h = decay * h + (delta * x)[..., None] * s["B"].float()[:, None]
    y = (h * s["C"].float()[:, None]).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * _sigmoid(z))
    if active is not None:
        y = torch.where(active[:, None], y, torch.zeros_like(y))
    return {"y": y.to(s["x"].dtype), "h_last": _put(s, s["h_last"], h, active, at)}


def _plain_norm_fwd(s):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    mean = None if s["case"]["rms"] else v.mean(1)
    c = v if mean is None else v - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + s["eps"])
    y = c * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype), "residual_out": None if s["residual"] is None else v.to(s["residual"].dtype),
            "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    dy, v = s["dy"].float(), s["v"].float()
    c = v if s["mean"] is None else v - s["mean"][:, None]
    xh = c * s["rstd"][:, None]
    g = dy * s["weight"]
    inner = g - xh * (g * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        inner = inner - g.mean(1, keepdim=True)
    dv = inner * s["rstd"][:, None]
    if s["dresidual_out"] is not None:
        dv = dv + s["dresidual_out"].float()
    return {"dx": dv.to(s["dy"].dtype), "dresidual": None if s["dresidual_out"] is None else dv.to(s["v"].dtype),
            "dweight": (dy.double() * xh.double()).sum(0).float(),
            "dbias": dy.double().sum(0).float() if s["bias"] is not None else None}


_plain = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
          "scan_step": _plain_scan_step, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}


def _own_conv_fwd(s):
    import selective_state_space_scan_amd as ssm
    y, last = ssm.causal_conv_fwd(s["x"], s["weight"], s["bias"], s["valid_len"], silu=s["case"]["silu"],
                                  conv0=s["conv0"])
    return {"y": y, "conv_last": last}


def _own_conv_bwd(s):
    import selective_state_space_scan_amd as ssm
    return ssm.causal_conv_bwd(s["x"], s["weight"], s["bias"], s["valid_len"], s["dy"], silu=s["case"]["silu"],
                               conv0=s["conv0"], dconv_last=s["dconv_last"])


def _own_conv_step(s):
    import selective_state_space_scan_amd as ssm
    y = ssm.causal_conv_step(s["x"], s["conv"], s["weight"], s["bias"], silu=s["case"]["silu"], slots=s["slots"],
                             conv_last=s["conv_last"], y=s["y"])
    return {"y": y, "conv_last": s["conv_last"]}


def _own_scan_step(s):
    import selective_state_space_scan_amd as ssm
    y = ssm.selective_scan_step(s["x"], s["delta"], s["A_log"], s["B"], s["C"], s["D"], s["h"],
                                delta_clamp=s["clamp"], delta_bias=s["delta_bias"], z=s["z"], slots=s["slots"],
                                h_last=s["h_last"], y=s["y"])
    return {"y": y, "h_last": s["h_last"]}


def _own_norm_fwd(s):
    import selective_state_space_scan_amd as ssm
    y, residual_out, mean, rstd = ssm.layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"],
                                                     eps=s["eps"], rms=s["case"]["rms"], return_stats=True)
    return {"y": y, "residual_out": residual_out, "mean": mean, "rstd": rstd}


def _own_norm_bwd(s):
    import selective_state_space_scan_amd as ssm
    return ssm.layer_norm_bwd(s["dy"], s["v"], s["weight"], s["mean"], s["rstd"], dresidual_out=s["dresidual_out"],
                              with_bias=s["bias"] is not None)


_own = {"conv_fwd": _own_conv_fwd, "conv_bwd": _own_conv_bwd, "conv_step": _own_conv_step,
        "scan_step": _own_scan_step, "norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd}


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    op, D = case["op"], case["dim"]
    e = 2 if case["io"] == "bf16" else 4
    if op in ("conv_fwd", "conv_bwd"):
        B, L, W = case["batch"], case["seqlen"], case["width"]
        n = B * L * D / (2 if case["ragged"] else 1)   # lengths are uniform in [0, L]: half of the steps are read
        edge = e * B * (W - 1) * D
        params = 4 * D * (W + (1 if case["bias"] else 0))
        if op == "conv_fwd":
            return {"bytes": int(e * (n + B * L * D) + edge * (2 if case["carry"] else 1) + params),
                    "flops": int(n * (2 * W + (4 if case["silu"] else 0)))}
        return {"bytes": int(e * (2 * n + B * L * D) + (3 * edge if case["carry"] else 0) + 2 * params),
                "flops": int(n * (4 * W + 1 + (2 * W + 8 if case["silu"] else 0)))}
    if op in ("conv_step", "scan_step"):
        B, live = case["batch"], case["batch"] - case["idle"]
        if op == "conv_step":
            W = case["width"]
            return {"bytes": int(e * D * (live * (2 * (W - 1) + 1) + B) + 4 * D * (W + (1 if case["bias"] else 0))
                                 + (4 * B if case["slots"] else 0)),
                    "flops": int(live * D * (2 * W + (4 if case["silu"] else 0)))}
        N = case["dstate"]
        ins = 2 + (1 if case["gate"] else 0)
        return {"bytes": int(8 * live * D * N + e * live * (ins * D + 2 * N) + e * B * D
                             + 4 * D * (N + 1 + (1 if case["skip"] else 0)) + (4 * B if case["slots"] else 0)),
                "flops": int(live * D * (7 * N + 8))}
    R = case["rows"]
    r = 4 if case["residual"] == "f32" else e
    has = case["residual"] != "none"
    params = 4 * D * (2 if case["bias"] else 1)
    stats = 4 * R * (1 if case["rms"] else 2)
    if op == "norm_fwd":
        return {"bytes": int(R * D * (2 * e + (2 * r if has else 0)) + params + stats), "flops": int(R * D * 9)}
    # one gradient serves x and the residual where both have one type
    return {"bytes": int(R * D * (2 * e + r + (r if has else 0) + (r if has and r != e else 0)) + 4 * D + params + stats),
            "flops": int(R * D * 14)}


# ---- the definition in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return _exact[case["op"]](case, s)


def _act(case, p):
    return p * torch.sigmoid(p) if case["silu"] else p


def _exact_conv_row(case, x, n, w, b, conv0):
    """(y, conv_last) of one row of n steps."""
    row = torch.cat([conv0, x[:n]])
    p = sum(row[k:k + n] * w[:, k] for k in range(w.shape[1]))
    if b is not None:
        p = p + b
    return torch.cat([_act(case, p), x.new_zeros((case["seqlen"] - n, x.shape[1]))]), row[n:]


def _exact_conv(case, s, x, w, b, conv0):
    lens = [case["seqlen"]] * case["batch"] if s["valid_len"] is None else s["valid_len"].tolist()
    rows = [_exact_conv_row(case, x[i], n, w, b, conv0[i]) for i, n in enumerate(lens)]
    return torch.stack([y for y, _ in rows]), torch.stack([last for _, last in rows])


def _exact_conv_fwd(case, s):
    conv0 = s["conv0"]
    if conv0 is None:
        conv0 = s["x"].new_zeros((case["batch"], case["width"] - 1, case["dim"]))
    y, last = _exact_conv(case, s, s["x"], s["weight"], s["bias"], conv0)
    return {"y": y, "conv_last": last}


def _exact_conv_bwd(case, s):
    """The derivative of the definition above, by reverse differentiation in 64 bits."""
    conv0 = s["conv0"]
    if conv0 is None:
        conv0 = s["x"].new_zeros((case["batch"], case["width"] - 1, case["dim"]))
    leaves = [t.detach().clone().requires_grad_() for t in (s["x"], s["weight"], conv0)]
    b = None if s["bias"] is None else s["bias"].detach().clone().requires_grad_()
    with torch.enable_grad():
        y, last = _exact_conv(case, s, leaves[0], leaves[1], b, leaves[2])
        # steps past a row's end have a constant output, and pass nothing back
        loss = (y * s["dy"]).sum()
        if s["dconv_last"] is not None:
            loss = loss + (last * s["dconv_last"]).sum()
        grads = torch.autograd.grad(loss, leaves + ([] if b is None else [b]), allow_unused=True)
    grads = [torch.zeros_like(t) if d is None else d for d, t in zip(grads, leaves + ([] if b is None else [b]))]
    return {"dx": grads[0], "dweight": grads[1], "dbias": None if b is None else grads[3],
            "dconv0": None if s["conv0"] is None else grads[2]}


def _exact_conv_step(case, s):
    y = torch.zeros_like(s["y"])
    last = s["conv_last"].clone()
    slots = range(case["batch"]) if s["slots"] is None else s["slots"].tolist()
    rows = [i for i, j in enumerate(slots) if j >= 0]
    at = [j for j in slots if j >= 0]
    old = s["conv"][at]
    p = s["x"][rows] * s["weight"][:, -1] + torch.einsum("bkd,dk->bd", old, s["weight"][:, :-1])
    if s["bias"] is not None:
        p = p + s["bias"]
    y[rows] = _act(case, p)
    last[at, :-1] = old[:, 1:]
    last[at, -1] = s["x"][rows]
    return {"y": y, "conv_last": last}


def _exact_scan_step(case, s):
    y = torch.zeros_like(s["y"])
    h_last = s["h_last"].clone()
    slots = range(case["batch"]) if s["slots"] is None else s["slots"].tolist()
    rows = [i for i, j in enumerate(slots) if j >= 0]
    at = [j for j in slots if j >= 0]
    delta = torch.logaddexp(s["delta"][rows] + s["delta_bias"], torch.zeros((), dtype=torch.float64, device=y.device))
    if s["clamp"] is not None:
        delta = delta.clip(*s["clamp"])
    x = s["x"][rows]
    h = s["h"][at] * torch.exp(delta.unsqueeze(2) * -s["A_log"].exp()) + torch.einsum("bd,bd,bn->bdn", delta, x, s["B"][rows])
    out = torch.einsum("bdn,bn->bd", h, s["C"][rows])
    if s["D"] is not None:
        out = out + x * s["D"]
    if s["z"] is not None:
        out = out * s["z"][rows] * torch.sigmoid(s["z"][rows])
    y[rows] = out
    h_last[at] = h
    return {"y": y, "h_last": h_last}


def _exact_norm_fwd(case, s):
    v = s["x"] if s["residual"] is None else s["x"] + s["residual"]
    if case["rms"]:
        mean, var = None, v.square().mean(1)
        c = v
    else:
        var, mean = torch.var_mean(v, 1, correction=0)
        c = v - mean[:, None]
    rstd = (var + s["eps"]).pow(-0.5)
    y = s["weight"] * (c * rstd[:, None])
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y, "residual_out": None if s["residual"] is None else v, "mean": mean, "rstd": rstd}


def _exact_norm_bwd(case, s):
    """From the Jacobian of the normalised row, r (I - 1 1^T / n - xh xh^T / n), the mean's part for layer norm alone."""
    r = s["rstd"][:, None]
    xh = s["v"] * r if s["mean"] is None else (s["v"] - s["mean"][:, None]) * r
    g = s["dy"] * s["weight"]
    n = case["dim"]
    along = torch.einsum("rd,rd->r", g, xh)[:, None] / n
    dv = r * g - r * along * xh
    if s["mean"] is not None:
        dv = dv - r * g.sum(1)[:, None] / n
    if s["dresidual_out"] is not None:
        dv = dv + s["dresidual_out"]
    return {"dx": dv, "dresidual": None if s["dresidual_out"] is None else dv,
            "dweight": torch.einsum("rd,rd->d", s["dy"], xh), "dbias": s["dy"].sum(0) if s["bias"] is not None else None}


_exact = {"conv_fwd": _exact_conv_fwd, "conv_bwd": _exact_conv_bwd, "conv_step": _exact_conv_step,
          "scan_step": _exact_scan_step, "norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd}
