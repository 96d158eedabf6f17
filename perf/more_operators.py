"""The gated recurrence and the group norm beside the selective scan: what is measured of them, and their plain forms.

Five directions of two operators, as a recurrent block uses them:

* ``rec_fwd``, ``rec_bwd``: the gated recurrence h = a h + sqrt(1 - a^2) sigmoid(x_gate) x with the decay
  a = exp(-exp(A_log) sigmoid(a_gate)), a state per channel, over whole sequences (prompts and training);
* ``rec_step``: the same for one token of every sequence, on the cache of states;
* ``gnorm_fwd``, ``gnorm_bwd``: the norm of each group of a step's channels behind it, with silu or a silu gate.

``run`` computes them from elementary torch operations in 32 bits, or, with ``own``, calls the framework.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64   # steps between the states that the forward keeps for the backward


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # A short float32 prompt: the smallest call, where latency counts.
        dict(name="rec_fwd-f32-b2-l256-d64", op="rec_fwd", io="f32", batch=2, seqlen=256, dim=64, wide=False, ragged=False,
             carry=False, states=False),
        # The forward of a training step at the scan's headline size, with the states that its backward takes.
        dict(name="rec_fwd-bf16-b8-l4096-d1024", op="rec_fwd", io="bf16", batch=8, seqlen=4096, dim=1024, wide=True,
             ragged=False, carry=False, states=True),
        # One long prompt, continued from its earlier part.
        dict(name="rec_fwd-bf16-b1-l32768-d2048", op="rec_fwd", io="bf16", batch=1, seqlen=32768, dim=2048, wide=True,
             ragged=False, carry=True, states=False),
        # An odd float32 training batch of sequences of different lengths, gradients through the carried states.
        dict(name="rec_bwd-f32-b3-l1021-d200", op="rec_bwd", io="f32", batch=3, seqlen=1021, dim=200, wide=False,
             ragged=True, carry=True),
        # A training step at the scan's headline size.
        dict(name="rec_bwd-bf16-b8-l4096-d1024", op="rec_bwd", io="bf16", batch=8, seqlen=4096, dim=1024, wide=True,
             ragged=False, carry=False),
        # A training step on long sequences of different lengths.
        dict(name="rec_bwd-bf16-b16-l8192-d512", op="rec_bwd", io="bf16", batch=16, seqlen=8192, dim=512, wide=False,
             ragged=True, carry=False),
        # One user's next token.
        dict(name="rec_step-bf16-b1-d2048", op="rec_step", io="bf16", batch=1, dim=2048, slots=0, idle=0),
        # The next token of a full serving batch, its sequences anywhere in a cache that holds twice as many.
        dict(name="rec_step-bf16-b256-d2048", op="rec_step", io="bf16", batch=256, dim=2048, slots=512, idle=3),
        # The norm behind the recurrence for a handful of sequences' next token, 8 groups of 125 channels.
        dict(name="gnorm_fwd-f32-r24-d1000-g8", op="gnorm_fwd", io="f32", rows=24, dim=1000, groups=8, rms=True, gate="none",
             silu=True, bias=False, wide=False),
        # The same over a training batch at the scan's headline size, gated by the block's other branch.
        dict(name="gnorm_fwd-bf16-r32768-d1024-g16", op="gnorm_fwd", io="bf16", rows=32768, dim=1024, groups=16, rms=False,
             gate="behind", silu=True, bias=True, wide=True),
        # An odd float32 training batch, 12 groups of 50 channels.
        dict(name="gnorm_bwd-f32-r1021-d600-g12", op="gnorm_bwd", io="f32", rows=1021, dim=600, groups=12, rms=False,
             gate="none", silu=True, bias=True, wide=False),
        # A training step at the scan's headline size, the gate in front of an RMS norm.
        dict(name="gnorm_bwd-bf16-r32768-d1024-g8", op="gnorm_bwd", io="bf16", rows=32768, dim=1024, groups=8, rms=True,
             gate="front", silu=True, bias=False, wide=True),
    ]


MAX_RECURRENT = 32768 * 2048   # elements of one [batch, length, dim] tensor of the recurrence's forward
MAX_ELEMENTS = 8 * 4096 * 1024   # of its backward, of the norms and of a cache


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A width: half of them multiples of 64, as models have them, the others anything."""
    d = _log_uniform(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["rec_fwd", "rec_bwd", "rec_step", "gnorm_fwd", "gnorm_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("rec_fwd", "rec_bwd"):
        most = MAX_ELEMENTS if op == "rec_bwd" or io == "f32" else MAX_RECURRENT
        dim = _dim(rng, 16, 4096)
        batch = _log_uniform(rng, 1, 16)
        seqlen = _log_uniform(rng, 1, max(1, min(32768, most // (dim * batch))))
        case = dict(op=op, io=io, batch=batch, seqlen=seqlen, dim=dim, wide=flip(), ragged=flip(), carry=flip())
        return dict(case, states=flip()) if op == "rec_fwd" else case
    if op == "rec_step":
        batch = _log_uniform(rng, 1, 512)
        slots = 2 * batch if flip() else 0
        return dict(op=op, io=io, batch=batch, dim=_dim(rng, 16, 8192), slots=slots,
                    idle=rng.randint(0, batch // 8) if slots else 0)
    size = _log_uniform(rng, 8, 1024)   # of a group: half of them multiples of 8, the others anything
    size = size // 8 * 8 if flip() else size
    groups = _log_uniform(rng, 1, max(1, 8192 // size))
    return dict(op=op, io=io, rows=_log_uniform(rng, 1, MAX_ELEMENTS // (groups * size)), dim=groups * size, groups=groups,
                rms=flip(), gate=rng.choice(["none", "behind", "front"]), silu=rng.random() < 0.8, bias=flip(), wide=flip())


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["io"]]
    dev = "cuda"

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device=dev) * scale + shift).to(dtype)

    s = dict(case=case)
    op, D = case["op"], case["dim"]
    if op in ("rec_fwd", "rec_bwd", "rec_step"):
        # at half-open gates a state decays by 1/e within 2 to 300 steps
        s["A_log"] = torch.rand(D, generator=g, device=dev) * 5.0 - 5.0
    if op in ("rec_fwd", "rec_bwd"):
        B, L = case["batch"], case["seqlen"]
        s["x"] = normal(B, L, D)
        if case["wide"]:   # both gates come out of one projection
            gates = normal(B, L, 2 * D)
            s["a_gate"], s["x_gate"] = gates[..., :D], gates[..., D:]
        else:
            s["a_gate"], s["x_gate"] = normal(B, L, D), normal(B, L, D)
        s["valid_len"] = (torch.randint(0, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
                          if case["ragged"] else None)
        s["h0"] = normal(B, D, dtype=torch.float32) if case["carry"] else None
        if op == "rec_bwd":
            s["dy"] = normal(B, L, D)
            s["dh_last"] = normal(B, D, dtype=torch.float32) if case["carry"] else None
            # what the forward kept: the state after every CHUNK steps
            states = torch.empty((B, -(-L // CHUNK), D), device=dev)
            h = torch.zeros((B, D), dtype=torch.float64, device=dev) if s["h0"] is None else s["h0"].double()
            n = torch.full((B,), L, device=dev) if s["valid_len"] is None else s["valid_len"].long()
            rate = torch.exp(s["A_log"].double())
            for c in range(states.shape[1]):
                at = slice(c * CHUNK, min(L, (c + 1) * CHUNK))
                left = (n[:, None] > torch.arange(at.start, at.stop, device=dev))[..., None]
                x, ag, xg = (s[k][:, at].double() for k in ("x", "a_gate", "x_gate"))
                d = torch.where(left, rate * torch.sigmoid(ag), 0.0)   # a padded step forgets nothing and adds nothing
                u = torch.where(left, torch.sqrt(-torch.expm1(-2 * d)) * torch.sigmoid(xg) * x, 0.0)
                past = torch.cumsum(d, 1)
                end = past[:, -1:]
                h = h * torch.exp(-end[:, 0]) + (u * torch.exp(past - end)).sum(1)
                states[:, c] = h
            s["chunk_states"] = states
            if case["wide"]:   # the gates' gradients go into the projection's
                dgates = torch.empty((B, L, 2 * D), dtype=dt, device=dev)
                s["da_gate"], s["dx_gate"] = dgates[..., :D], dgates[..., D:]
            else:
                s["da_gate"] = s["dx_gate"] = None
    elif op == "rec_step":
        B = case["batch"]
        n = case["slots"] or B
        s["slots"] = None
        if case["slots"]:
            slots = torch.randperm(n, generator=g, device=dev)[:B].to(torch.int32)
            if case["idle"]:
                slots[B - case["idle"]:] = -1   # rows that pad the batch
            s["slots"] = slots
        s["x"] = normal(B, D)
        gates = normal(B, 2 * D)
        s["a_gate"], s["x_gate"] = gates[:, :D], gates[:, D:]
        s["h"] = normal(n, D, dtype=torch.float32)
        s["h_last"] = torch.zeros_like(s["h"])
        s["y"] = torch.empty((B, D), dtype=dt, device=dev)
    else:
        R, G = case["rows"], case["groups"]
        s["eps"] = 1e-5
        s["weight"] = normal(D, dtype=torch.float32, scale=0.1, shift=1.0)
        s["bias"] = normal(D, dtype=torch.float32, scale=0.1) if case["bias"] else None
        s["x"] = normal(R, D, scale=2.0, shift=0.3)
        s["z"] = None if case["gate"] == "none" else (normal(R, 2 * D)[:, D:] if case["wide"] else normal(R, D))
        if op == "gnorm_bwd":
            s["dy"] = normal(R, D)
            v = s["x"].double()
            if case["gate"] == "front":
                z = s["z"].double()
                v = v * (z * torch.sigmoid(z) if case["silu"] else z)
            v = v.view(R, G, D // G)
            mean = torch.zeros((R, G), dtype=torch.float64, device=dev) if case["rms"] else v.mean(2)
            s["rstd"] = (((v - mean[..., None]) ** 2).mean(2) + s["eps"]).rsqrt().float()
            s["mean"] = None if case["rms"] else mean.float()
            # the gate's gradient goes into its projection's
            s["dz"] = torch.empty((R, 2 * D), dtype=dt, device=dev)[:, D:] if case["wide"] and s["z"] is not None else None
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _scan(a, u):
    """h[t] = a[t] h[t-1] + u[t] along dimension 1, by doubling."""
    step = 1
    while step < u.shape[1]:
        u = torch.cat([u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return u


def _valid(s):
    """Which steps are valid, [batch, length, 1]."""
    B, L, _ = s["x"].shape
    t = torch.arange(L, device=s["x"].device)
    n = torch.full((B,), L, device=t.device) if s["valid_len"] is None else s["valid_len"].long().clamp(0, L)
    return (t[None, :] < n[:, None])[..., None]


def _gates(s, valid=None):
    """Both gates and the decay's exponent and the input's scale, in 32 bits; a padded step forgets nothing and adds
    nothing."""
    r, i = _sigmoid(s["a_gate"].float()), _sigmoid(s["x_gate"].float())
    d = torch.exp(s["A_log"]) * r
    if valid is not None:
        d = torch.where(valid, d, torch.zeros_like(d))
    return r, i, d, torch.sqrt(-torch.expm1(-2 * d))


def _start(s):
    return s["x"].new_zeros((s["x"].shape[0], s["x"].shape[2]), dtype=torch.float32) if s["h0"] is None else s["h0"]


def _plain_rec_fwd(s):
    valid = _valid(s)
    r, i, d, scale = _gates(s, valid)
    u = torch.where(valid, scale * i * s["x"].float(), torch.zeros_like(d))
    h = _scan(torch.cat([torch.ones_like(d[:, :1]), torch.exp(-d)], 1), torch.cat([_start(s)[:, None], u], 1))[:, 1:]
    y = torch.where(valid, h, torch.zeros_like(h)).to(s["x"].dtype)
    ends = torch.arange(CHUNK, h.shape[1] + CHUNK, CHUNK, device=h.device).clamp(max=h.shape[1]) - 1
    return {"y": y, "h_last": h[:, -1].clone(), "chunk_states": h[:, ends] if s["case"]["states"] else None}


def _plain_rec_bwd(s):
    valid = _valid(s)
    dt = s["x"].dtype
    r, i, d, scale = _gates(s, valid)
    a = torch.exp(-d)
    x = torch.where(valid, s["x"].float(), torch.zeros_like(d))
    u = scale * i * x
    # the states again, each chunk from the one that the forward kept before it
    B, L, D = x.shape
    C = s["chunk_states"].shape[1]
    first = torch.cat([_start(s)[:, None], s["chunk_states"][:, :-1]], 1)[:, :, None]
    cut = lambda t: torch.cat([t, t.new_zeros((B, C * CHUNK - L, D))], 1).view(B, C, CHUNK, D)  # noqa: E731
    us, as_ = torch.cat([first, cut(u)], 2), torch.cat([torch.ones_like(first), cut(a)], 2)
    h = _scan(as_.view(B * C, CHUNK + 1, D), us.view(B * C, CHUNK + 1, D))[:, :CHUNK].reshape(B, C * CHUNK, D)[:, :L]
    # g: the gradient of every step's state, from the last step back
    g = torch.where(valid, s["dy"].float(), torch.zeros_like(x))
    if s["dh_last"] is not None:
        g = torch.cat([g[:, :-1], g[:, -1:] + s["dh_last"][:, None]], 1)
    g = _scan(torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1), g.flip(1)).flip(1)
    # d's own gradient times d; d a^2 / scale goes to 0 with d
    ratio = torch.where(d > 0, d * a * a / scale, torch.zeros_like(d))
    q = ratio * g * i * x - d * a * g * h
    grads = {"dx": g * scale * i, "da_gate": q * (1 - r), "dx_gate": g * u * (1 - i)}
    grads = {k: torch.where(valid, v, torch.zeros_like(v)).to(s["x"].dtype) for k, v in grads.items()}
    return dict(grads, dA_log=q.double().sum((0, 1)).float(), dh0=a[:, 0] * g[:, 0] if s["h0"] is not None else None)


def _plain_rec_step(s):
    h, at = s["h"], None
    if s["slots"] is not None:
        at = s["slots"].long()
        h = h[at.clamp(min=0)]
    r, i, d, scale = _gates(s)
    h = torch.exp(-d) * h + scale * i * s["x"].float()
    y = h
    if at is None:
        s["h_last"].copy_(h)
    else:
        y = torch.where((at >= 0)[:, None], h, torch.zeros_like(h))
        # the idle rows write a spare row behind the cache
        ext = torch.cat([s["h_last"], h[:1]])
        ext[torch.where(at >= 0, at, torch.full_like(at, s["h"].shape[0]))] = h
        s["h_last"].copy_(ext[:-1])
    return {"y": y.to(s["x"].dtype), "h_last": s["h_last"]}


def _act(case, u):
    """The activation, and its derivative."""
    if not case["silu"]:
        return u, torch.ones_like(u)
    sg = _sigmoid(u)
    return u * sg, sg * (1 + u * (1 - sg))


def _normed(s):
    """What is normalised, [rows, groups, size]."""
    case, v = s["case"], s["x"].float()
    if case["gate"] == "front":
        v = v * _act(case, s["z"].float())[0]
    return v.view(case["rows"], case["groups"], -1)


def _plain_gnorm_fwd(s):
    case = s["case"]
    v = _normed(s)
    mean = None if case["rms"] else v.mean(2)
    c = v if mean is None else v - mean[..., None]
    rstd = 1 / torch.sqrt((c * c).mean(2) + s["eps"])
    p = (c * rstd[..., None]).view(s["x"].shape) * s["weight"]
    if s["bias"] is not None:
        p = p + s["bias"]
    if case["gate"] == "none":
        p = _act(case, p)[0]
    elif case["gate"] == "behind":
        p = p * _act(case, s["z"].float())[0]
    return {"y": p.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_gnorm_bwd(s):
    case, dt = s["case"], s["x"].dtype
    v = _normed(s)
    xh = (v if s["mean"] is None else v - s["mean"][..., None]) * s["rstd"][..., None]
    flat = xh.view(s["x"].shape)
    p = flat * s["weight"]
    if s["bias"] is not None:
        p = p + s["bias"]
    dp, dz = s["dy"].float(), None
    if case["gate"] == "none":
        dp = dp * _act(case, p)[1]
    elif case["gate"] == "behind":
        act, slope = _act(case, s["z"].float())
        dz = dp * p * slope
        dp = dp * act
    gr = (dp * s["weight"]).view(v.shape)
    dv = gr - xh * (gr * xh).mean(2, keepdim=True)
    if s["mean"] is not None:
        dv = dv - gr.mean(2, keepdim=True)
    dx = (dv * s["rstd"][..., None]).view(flat.shape)
    if case["gate"] == "front":
        act, slope = _act(case, s["z"].float())
        dz = dx * s["x"].float() * slope
        dx = dx * act
    return {"dx": dx.to(dt), "dz": None if dz is None else dz.to(dt),
            "dweight": (dp.double() * flat.double()).sum(0).float(),
            "dbias": None if s["bias"] is None else dp.double().sum(0).float()}


_plain = {"rec_fwd": _plain_rec_fwd, "rec_bwd": _plain_rec_bwd, "rec_step": _plain_rec_step,
          "gnorm_fwd": _plain_gnorm_fwd, "gnorm_bwd": _plain_gnorm_bwd}


def _own_rec_fwd(s):
    import selective_state_space_scan_amd as ssm
    out = ssm.gated_recurrence_fwd(s["x"], s["a_gate"], s["x_gate"], s["A_log"], s["valid_len"], h0=s["h0"],
                                   return_chunk_states=s["case"]["states"])
    return {"y": out[0], "h_last": out[1], "chunk_states": out[2] if s["case"]["states"] else None}


def _own_rec_bwd(s):
    import selective_state_space_scan_amd as ssm
    return ssm.gated_recurrence_bwd(s["x"], s["a_gate"], s["x_gate"], s["A_log"], s["valid_len"], s["dy"],
                                    s["chunk_states"], h0=s["h0"], dh_last=s["dh_last"], da_gate=s["da_gate"],
                                    dx_gate=s["dx_gate"])


def _own_rec_step(s):
    import selective_state_space_scan_amd as ssm
    y = ssm.gated_recurrence_step(s["x"], s["a_gate"], s["x_gate"], s["A_log"], s["h"], slots=s["slots"],
                                  h_last=s["h_last"], y=s["y"])
    return {"y": y, "h_last": s["h_last"]}


def _own_gnorm_fwd(s):
    import selective_state_space_scan_amd as ssm
    case = s["case"]
    y, mean, rstd = ssm.group_norm_fwd(s["x"], case["groups"], s["weight"], s["bias"], z=s["z"], silu=case["silu"],
                                       gate_first=case["gate"] == "front", eps=s["eps"], rms=case["rms"],
                                       return_stats=True)
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_gnorm_bwd(s):
    import selective_state_space_scan_amd as ssm
    case = s["case"]
    return ssm.group_norm_bwd(s["dy"], s["x"], case["groups"], s["weight"], s["bias"], s["mean"], s["rstd"], z=s["z"],
                              silu=case["silu"], gate_first=case["gate"] == "front", dz=s["dz"])


_own = {"rec_fwd": _own_rec_fwd, "rec_bwd": _own_rec_bwd, "rec_step": _own_rec_step,
        "gnorm_fwd": _own_gnorm_fwd, "gnorm_bwd": _own_gnorm_bwd}


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    op, D = case["op"], case["dim"]
    e = 2 if case["io"] == "bf16" else 4
    if op in ("rec_fwd", "rec_bwd"):
        B, L = case["batch"], case["seqlen"]
        n = B * L * D / (2 if case["ragged"] else 1)   # lengths are uniform in [0, L]: half of the steps are read
        state, kept = 4 * B * D, 4 * B * D * (-(-L // CHUNK))
        if op == "rec_fwd":
            return {"bytes": int(e * (3 * n + B * L * D) + state * (2 if case["carry"] else 1)
                                 + (kept if case["states"] else 0) + 4 * D), "flops": int(n * 20)}
        return {"bytes": int(e * (4 * n + 3 * B * L * D) + kept + (3 * state if case["carry"] else 0) + 8 * D),
                "flops": int(n * 45)}
    if op == "rec_step":
        B, live = case["batch"], case["batch"] - case["idle"]
        return {"bytes": int(live * D * (8 + 3 * e) + e * B * D + 4 * D + (4 * B if case["slots"] else 0)),
                "flops": int(live * D * 20)}
    R, gated = case["rows"], case["gate"] != "none"
    params = 4 * D * (2 if case["bias"] else 1)
    stats = 4 * R * case["groups"] * (1 if case["rms"] else 2)
    act = 5 if case["silu"] else 0
    if op == "gnorm_fwd":
        return {"bytes": int(R * D * e * (3 if gated else 2) + params + stats), "flops": int(R * D * (9 + act))}
    return {"bytes": int(R * D * e * (5 if gated else 3) + 2 * params + stats), "flops": int(R * D * (16 + 2 * act))}


# ---- the definition in 64 bits ---------------------------------------------

def exact(case, seed):
    """Step after step in 64 bits; gradients by reverse differentiation of that."""
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]

    def grads(out, seeds, leaves):
        got = torch.autograd.grad(sum((o * d).sum() for o, d in zip(out, seeds) if d is not None), leaves, allow_unused=True)
        return [torch.zeros_like(t) if d is None else d for d, t in zip(got, leaves)]

    def advance(h, x, ag, xg, A_log):
        forget = torch.exp(-A_log.exp() * ag.sigmoid())
        return forget * h + (1 - forget.square()).sqrt() * xg.sigmoid() * x

    if op in ("rec_fwd", "rec_bwd"):
        B, L, D = s["x"].shape
        lens = torch.full((B,), L, device="cuda") if s["valid_len"] is None else s["valid_len"]
        left = lens[:, None] > torch.arange(L, device="cuda")
        h0 = s["x"].new_zeros((B, D)) if s["h0"] is None else s["h0"]
        leaves = [s["x"], s["a_gate"], s["x_gate"], s["A_log"], h0]
        if op == "rec_bwd":
            leaves = [t.detach().clone().requires_grad_() for t in leaves]
        x, ag, xg, A_log, h0 = leaves
        with torch.set_grad_enabled(op == "rec_bwd"):
            forget = torch.exp(-A_log.exp() * ag.sigmoid())
            put = (1 - forget.square()).sqrt() * xg.sigmoid() * x
            # a padded step leaves the state as it is
            forget, put = torch.where(left[..., None], forget, 1.0), torch.where(left[..., None], put, 0.0)
            h, hs = h0, []
            for f, p in zip(forget.unbind(1), put.unbind(1)):
                h = torch.addcmul(p, f, h)
                hs.append(h)
            y = torch.where(left[..., None], torch.stack(hs, 1), 0.0)
            if op == "rec_fwd":
                kept = torch.stack([hs[min(t, L) - 1] for t in range(CHUNK, L + CHUNK, CHUNK)], 1) if case["states"] else None
                return {"y": y, "h_last": h, "chunk_states": kept}
            dx, da, dxg, dA, dh0 = grads([y, h], [s["dy"], s["dh_last"]], leaves)
        return {"dx": dx, "da_gate": da, "dx_gate": dxg, "dA_log": dA, "dh0": None if s["h0"] is None else dh0}

    if op == "rec_step":
        y, h_last = torch.zeros_like(s["y"]), s["h_last"].clone()
        slots = list(range(case["batch"])) if s["slots"] is None else s["slots"].tolist()
        rows = [b for b, j in enumerate(slots) if j >= 0]
        at = [slots[b] for b in rows]
        y[rows] = h_last[at] = advance(s["h"][at], s["x"][rows], s["a_gate"][rows], s["x_gate"][rows], s["A_log"])
        return {"y": y, "h_last": h_last}

    R, G = case["rows"], case["groups"]
    act = torch.nn.functional.silu if case["silu"] else (lambda u: u)
    zero = s["x"].new_zeros(case["dim"])
    leaves = [s["x"], s["weight"], zero if s["bias"] is None else s["bias"]] + ([] if s["z"] is None else [s["z"]])
    if op == "gnorm_bwd":
        leaves = [t.detach().clone().requires_grad_() for t in leaves]
    with torch.set_grad_enabled(op == "gnorm_bwd"):
        x, w, b = leaves[:3]
        v = (x * act(leaves[3]) if case["gate"] == "front" else x).reshape(R, G, -1)
        if case["rms"]:
            mean, var, c = None, v.square().mean(2), v
        else:
            var, mean = torch.var_mean(v, 2, correction=0)
            c = v - mean[..., None]
        rstd = (var + s["eps"]).pow(-0.5)
        y = (c * rstd[..., None]).reshape(R, -1) * w + b
        y = act(y) if case["gate"] == "none" else y * act(leaves[3]) if case["gate"] == "behind" else y
        if op == "gnorm_fwd":
            return {"y": y, "mean": mean, "rstd": rstd}
        got = grads([y], [s["dy"]], leaves)
    return {"dx": got[0], "dz": None if s["z"] is None else got[3], "dweight": got[1],
            "dbias": None if s["bias"] is None else got[2]}
