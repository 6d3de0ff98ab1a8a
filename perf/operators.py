"""What is measured of the recurrent block's operators: the gated linear recurrence and the layer norm.

Gated linear recurrence over [B, L, D] (one state per channel), with s_t = sigmoid(gate_t):

    without a rate:      a_t = s_t,                beta_t = 1 - s_t
    with rate[d] > 0:    a_t = exp(-rate[d] s_t),  beta_t = sqrt(1 - a_t^2)
    h_t = a_t h_{t-1} + beta_t sigmoid(input_gate_t) x_t   (no input gate: factor 1),   y_t = h_t

Layer norm over the last axis of [rows, D], after an optional residual addition whose sum is rounded to the
residual's type and kept:

    s = x + residual,   y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias     (rms: no mean is removed)

Sizes are those of this repository's workloads (1536, 2048, 4096 and 5120 channels, 131072 tokens, 256 decoded
sequences) and odd ones.
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------------------------------------- cases

def _glr(name, op, B, L, D, dtype, decay, input_gate, state):
    return {"name": name, "op": op, "B": B, "L": L, "D": D, "dtype": dtype, "decay": decay,
            "input_gate": input_gate, "state": state}


def _norm(name, op, rows, D, dtype, residual, rms, bias):
    return {"name": name, "op": op, "rows": rows, "D": D, "dtype": dtype, "residual": residual, "rms": rms,
            "bias": bias}


def listed():
    return [
        # one generated token of one sequence: latency
        _glr("recurrence step, 1 row", "glr_step", 1, 1, 2048, "bf16", True, True, True),
        # one generated token of a served batch
        _glr("recurrence step, 256 rows", "glr_step", 256, 1, 2048, "f32", False, False, True),
        # a prompt of odd length and width, continued from a state
        _glr("recurrence, odd sizes", "glr_forward", 3, 1001, 515, "bf16", True, False, True),
        # the forward pass of an ordinary batch
        _glr("recurrence, 8 x 2048", "glr_forward", 8, 2048, 1536, "f32", False, False, False),
        # a long document
        _glr("recurrence, 131072 tokens", "glr_forward", 1, 131072, 2048, "bf16", True, True, True),
        # training steps: the forward pass and all gradients
        _glr("recurrence train, odd sizes", "glr_train", 3, 777, 201, "f32", True, True, True),
        _glr("recurrence train, 8 x 2048", "glr_train", 8, 2048, 1536, "bf16", True, True, False),
        _glr("recurrence train, 2 x 8192", "glr_train", 2, 8192, 4096, "bf16", False, False, True),
        # the norm before a block: one generated token, a long prompt with the residual stream in fp32
        _norm("norm, 1 row", "norm_forward", 1, 2048, "bf16", "same", False, True),
        _norm("norm, 32768 rows", "norm_forward", 32768, 2048, "bf16", "f32", True, False),
        # training steps of the norm
        _norm("norm train, odd sizes", "norm_train", 2001, 777, "f32", "none", False, True),
        _norm("norm train, 16384 rows", "norm_train", 16384, 5120, "bf16", "same", False, True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr_step", "glr_forward", "glr_forward", "glr_train", "glr_train", "norm_forward", "norm_train"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("norm"):
        D = _spread(rng, 64, 8192)
        D = D if rng.random() < 0.3 else D // 16 * 16
        rows = _spread(rng, 1, min(65536, (1 << 26) // D))
        c = _norm("", op, rows, D, dtype, rng.choice(["none", "same", "f32"]), rng.random() < 0.5, rng.random() < 0.5)
    else:
        D = _spread(rng, 64, 8192)
        D = D if rng.random() < 0.3 else D // 8 * 8
        B = _spread(rng, 1, 512 if op == "glr_step" else 16)
        most = (1 << 26) if op == "glr_forward" else (1 << 25)
        L = _spread(rng, 1, 4) if op == "glr_step" else _spread(rng, 2, min(131072, most // (B * D)))
        c = _glr("", op, B, L, D, dtype, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.6)
    del c["name"]
    return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, D = case["rows"], case["D"]
        rt = torch.float32 if case["residual"] == "f32" else dt
        s["x"] = normal(rows, D)
        s["residual"] = None if case["residual"] == "none" else normal(rows, D, std=2.0, dtype=rt)
        s["weight"] = normal(D, mean=1.0, std=0.1, dtype=torch.float32)
        s["bias"] = normal(D, std=0.1, dtype=torch.float32) if case["bias"] else None
        if case["op"] == "norm_train":
            s["dy"] = normal(rows, D)
            s["dresidual"] = None if case["residual"] == "none" else normal(rows, D, dtype=rt)
        return s
    B, L, D = case["B"], case["L"], case["D"]
    s["x"] = normal(B, L, D)
    # open forget gates without a rate (a around 0.9); with one, half-open gates and decays per token from
    # exp(-0.4) to exp(-0.004)
    s["gate"] = normal(B, L, D) if case["decay"] else normal(B, L, D, mean=2.0)
    s["rate"] = None
    if case["decay"]:
        u = torch.rand(D, generator=g, device="cuda")
        s["rate"] = torch.exp(math.log(0.008) + u * (math.log(0.8) - math.log(0.008)))
    s["input_gate"] = normal(B, L, D) if case["input_gate"] else None
    s["h0"] = normal(B, D, dtype=torch.float32) if case["state"] else None
    if case["op"] == "glr_train":
        s["dy"] = normal(B, L, D)
        s["dh_final"] = normal(B, D, dtype=torch.float32) if case["state"] else None
    return s


# ------------------------------------------------------------------------------------------------- plain forms

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1, by doubling: after the round of span k, (a, b) at t is the composition
    of the last 2k maps.  log2(L) rounds; there is no elementary torch operation that scans affine maps."""
    k, L = 1, a.shape[1]
    while k < L:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _gates(s):
    """sigmoid(gate), 1 - sigmoid(gate), the decay a, beta, sigmoid(input gate) (or 1), x: all in 32 bits."""
    x, g = s["x"].float(), s["gate"].float()
    sg, sn = torch.sigmoid(g), torch.sigmoid(-g)
    if s["rate"] is None:
        a, beta = sg, sn
    else:
        z = sg * s["rate"]
        a, beta = torch.exp(-z), torch.sqrt(-torch.expm1(-2 * z))
    si = 1.0 if s["input_gate"] is None else torch.sigmoid(s["input_gate"].float())
    return sg, sn, a, beta, si, x


def _plain_glr_forward(s):
    _, _, a, beta, si, x = _gates(s)
    b = beta * (si * x)
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, b)
    return h


def _plain_glr_backward(s, h):
    sg, sn, a, beta, si, x = _gates(s)
    dt = s["x"].dtype
    h0 = torch.zeros_like(h[:, 0]) if s["h0"] is None else s["h0"]
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    dy = s["dy"].float()
    if s["dh_final"] is not None:
        dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dh_final"][:, None]], 1)
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    G = _scan(later.flip(1), dy.flip(1)).flip(1)
    out = {"dx": (G * beta * si).to(dt), "dh0": a[:, 0] * G[:, 0]}
    if s["input_gate"] is not None:
        out["dinput_gate"] = (G * beta * x * si * torch.sigmoid(-s["input_gate"].float())).to(dt)
    if s["rate"] is None:
        out["dgate"] = (G * (before - si * x) * sg * sn).to(dt)
    else:
        q = G * a * (before - a / beta * si * x)
        out["dgate"] = (-q * s["rate"] * sg * sn).to(dt)
        out["drate"] = -(q * sg).sum((0, 1))
    return out


def _plain_norm_forward(s):
    rms = s["case"]["rms"]
    t = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = t.float()
    mean = 0.0 if rms else v.mean(1, keepdim=True)
    rstd = torch.rsqrt(((v - mean) ** 2).mean(1, keepdim=True) + EPS)
    y = (v - mean) * rstd * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype), t, mean, rstd


def _plain_norm_backward(s, t, mean, rstd):
    xhat = (t.float() - mean) * rstd
    dy = s["dy"].float()
    wdy = dy * s["weight"]
    d = wdy - xhat * (wdy * xhat).mean(1, keepdim=True)
    if not s["case"]["rms"]:
        d = d - wdy.mean(1, keepdim=True)
    d = d * rstd
    if s["dresidual"] is not None:
        d = d + s["dresidual"].float()
    out = {"dx": d.to(s["x"].dtype), "dweight": (dy * xhat).sum(0)}
    if s["residual"] is not None:
        out["dresidual"] = d.to(s["residual"].dtype)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


# ------------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op.startswith("norm"):
        return _norm_pass(s, op == "norm_train")
    return _glr_pass(s, op == "glr_train")


def _glr_pass(s, train):
    if own:
        from selective_state_space_32_b200 import sscan
        y, h_final, states = sscan.glr_forward(s["x"], s["gate"], rate=s["rate"], input_gate=s["input_gate"],
                                               h0=s["h0"], want_states=train)
        out = {"y": y, "h_final": h_final}
        if train:
            d = sscan.glr_backward(s["x"], s["gate"], s["dy"], states, rate=s["rate"], input_gate=s["input_gate"],
                                   dh_final=s["dh_final"])
            out.update((k, v) for k, v in d.items() if v is not None)
        return out
    h = _plain_glr_forward(s)
    out = {"y": h.to(s["x"].dtype), "h_final": h[:, -1].clone()}
    if train:
        out.update(_plain_glr_backward(s, h))
    return out


def _norm_pass(s, train):
    rms = s["case"]["rms"]
    if own:
        from selective_state_space_32_b200 import sscan
        y, t, mean, rstd = sscan.norm_forward(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS, rms=rms,
                                              want_stats=train)
        out = {"y": y} if s["residual"] is None else {"y": y, "residual_out": t}
        if train:
            d = sscan.norm_backward(s["dy"], t, mean, rstd, s["weight"], dresidual=s["dresidual"], rms=rms,
                                    want_dbias=s["bias"] is not None)
            out.update((k, v) for k, v in d.items() if v is not None and (k != "dresidual" or s["residual"] is not None))
        return out
    y, t, mean, rstd = _plain_norm_forward(s)
    out = {"y": y} if s["residual"] is None else {"y": y, "residual_out": t}
    if train:
        out.update(_plain_norm_backward(s, t, mean, rstd))
    return out


# ------------------------------------------------------------------------------------------------- floors

def work(case):
    """Every input read once, every output written once; the operations of the formulas."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, D = case["rows"] * case["D"], case["D"]
        r = {"none": 0, "same": e, "f32": 4}[case["residual"]]
        params = 4 * D * (2 if case["bias"] else 1)
        if case["op"] == "norm_forward":
            return {"bytes": n * (2 * e + 2 * r) + params, "flops": 9 * n}
        # x, residual, dy, dresidual in; y, the sum, dx, dresidual out
        return {"bytes": n * (4 * e + 4 * r) + 2 * params, "flops": 22 * n}
    n, bd = case["B"] * case["L"] * case["D"], case["B"] * case["D"]
    gates = 2 if case["input_gate"] else 1
    per = (12 if case["decay"] else 8) + (4 if case["input_gate"] else 0)
    small = 4 * bd * (2 if case["state"] else 1) + (4 * case["D"] if case["decay"] else 0)
    if case["op"] != "glr_train":
        return {"bytes": n * e * (2 + gates) + small, "flops": per * n}
    # x, the gates, dy in; y, dx, the gates' gradients out; h0, dh_final in, h_final, dh0 out
    return {"bytes": n * e * (4 + 2 * gates) + 2 * small, "flops": 3 * per * n}


# ------------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    return _exact_norm(case, s, d) if case["op"].startswith("norm") else _exact_glr(case, d)


def _exact_glr(case, d):
    """Token by token, from the definition; the gradients by the chain rule of one token's update, last token first."""
    B, L, D = case["B"], case["L"], case["D"]
    if (L > 300000) or B * L * D > 1 << 28:
        return None
    x, c = d["x"], d["rate"]
    sig = 1 / (1 + torch.exp(-d["gate"]))
    if c is None:
        a = sig
        beta = 1 / (1 + torch.exp(d["gate"]))
    else:
        a = torch.exp(-c * sig)
        beta = torch.sqrt((1 - a) * (1 + a))
    inp = x if d["input_gate"] is None else x / (1 + torch.exp(-d["input_gate"]))
    h = torch.zeros(B, D, dtype=torch.float64, device="cuda") if d["h0"] is None else d["h0"].clone()
    hs = beta * inp
    for t in range(L):
        h = hs[:, t].addcmul_(a[:, t], h)
    out = {"y": hs, "h_final": h.clone()}
    if case["op"] != "glr_train":
        return out
    prev = torch.empty_like(hs)
    prev[:, 1:] = hs[:, :-1]
    prev[:, 0] = 0.0 if d["h0"] is None else d["h0"]
    G = d["dy"].clone()
    carry = torch.zeros(B, D, dtype=torch.float64, device="cuda") if d["dh_final"] is None else d["dh_final"]
    for t in range(L - 1, -1, -1):
        carry = G[:, t].add_(carry) * a[:, t]
    out["dh0"] = carry
    dinp = G * beta
    if d["input_gate"] is None:
        out["dx"] = dinp
    else:
        si = 1 / (1 + torch.exp(-d["input_gate"]))
        out["dx"] = dinp * si
        out["dinput_gate"] = dinp * x * si * (1 - si)
    # d h_t / d a_t through the decay and through beta
    da = G * (prev - inp) if c is None else G * (prev - inp * a / beta)
    if c is None:
        out["dgate"] = da * sig * (1 - sig)
    else:
        ds = da * a * -c
        out["dgate"] = ds * sig * (1 - sig)
        out["drate"] = (da * a * -sig).sum(1).sum(0)
    return out


def _exact_norm(case, s, d):
    t = d["x"]
    if d["residual"] is not None:
        t = (d["x"] + d["residual"]).to(s["residual"].dtype).double()
    n = case["D"]
    mu = torch.zeros_like(t[:, :1]) if case["rms"] else t.sum(1, keepdim=True) / n
    sd = torch.sqrt((t - mu).square().sum(1, keepdim=True) / n + EPS)
    z = (t - mu) / sd
    y = z * d["weight"] + (0.0 if d["bias"] is None else d["bias"])
    out = {"y": y} if d["residual"] is None else {"y": y, "residual_out": t}
    if case["op"] == "norm_forward":
        return out
    dz = d["dy"] * d["weight"]
    g = dz - z * ((dz * z).sum(1, keepdim=True) / n)
    if not case["rms"]:
        g = g - dz.sum(1, keepdim=True) / n
    g = g / sd
    if d["dresidual"] is not None:
        g = g + d["dresidual"]
    out["dx"] = g
    out["dweight"] = (d["dy"] * z).sum(0)
    if d["residual"] is not None:
        out["dresidual"] = g
    if d["bias"] is not None:
        out["dbias"] = d["dy"].sum(0)
    return out
