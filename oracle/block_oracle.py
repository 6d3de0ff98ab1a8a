"""Oracle of the recurrent block's operators in fp64 (numpy): the gated linear recurrence
and the layer norm, forward and backward, from their definitions.

Gated linear recurrence, per batch row and channel, s = sigmoid(gate), u = sigmoid(input_gate) x:

    no rate: a = s, beta = 1 - s;   rate c: a = exp(-c s), beta = sqrt(1 - a^2)
    h_t = a_t h_{t-1} + beta_t u_t,  y_t = h_t

Layer norm: z = (s - mean) rstd, y = z w + b (rms: mean = 0).

The gradients are written token by token and row by row from the chain rule; they are
pinned by central differences of the forward functions.  Shares no code with the CUDA path.
"""
import numpy as np


def _sig(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def _f64(a):
    return None if a is None else np.asarray(a, np.float64)


def glr_coefficients(gate, rate=None):
    """(a, beta) of every token."""
    s = _sig(_f64(gate))
    if rate is None:
        return s, _sig(-_f64(gate))
    z = _f64(rate) * s
    return np.exp(-z), np.sqrt(-np.expm1(-2.0 * z))


def glr_forward(x, gate, rate=None, input_gate=None, h0=None):
    """x, gate, input_gate: [B, L, D]; rate [D]; h0 [B, D].  Returns (y [B, L, D], h_final [B, D])."""
    x = _f64(x)
    B, L, D = x.shape
    a, beta = glr_coefficients(gate, rate)
    u = x if input_gate is None else x * _sig(_f64(input_gate))
    h = np.zeros((B, D)) if h0 is None else _f64(h0).copy()
    y = np.empty((B, L, D))
    for t in range(L):
        h = a[:, t] * h + beta[:, t] * u[:, t]
        y[:, t] = h
    return y, h


def glr_backward(x, gate, dy, rate=None, input_gate=None, h0=None, dh_final=None):
    """Gradients given dy and dh_final: dict of dx, dgate, dinput_gate, drate, dh0 (and G, the
    whole gradient of every h_t, and prev, the state before every token, for error bounds)."""
    x, gate, dy = _f64(x), _f64(gate), _f64(dy)
    B, L, D = x.shape
    a, beta = glr_coefficients(gate, rate)
    s, n = _sig(gate), _sig(-gate)
    si = np.ones_like(x) if input_gate is None else _sig(_f64(input_gate))
    u = x * si
    y, _ = glr_forward(x, gate, rate, input_gate, h0)
    prev = np.empty_like(y)
    prev[:, 1:] = y[:, :-1]
    if L:
        prev[:, 0] = 0.0 if h0 is None else h0
    G = np.empty_like(y)
    carry = np.zeros((B, D)) if dh_final is None else _f64(dh_final).copy()
    for t in range(L - 1, -1, -1):
        G[:, t] = dy[:, t] + carry
        carry = a[:, t] * G[:, t]
    out = {"dx": G * beta * si, "dinput_gate": None, "drate": None, "dh0": carry, "G": G, "prev": prev}
    if input_gate is not None:
        out["dinput_gate"] = G * beta * x * si * _sig(-_f64(input_gate))
    if rate is None:
        out["dgate"] = G * (prev - u) * s * n
    else:
        with np.errstate(divide="ignore", invalid="ignore"):
            ratio = np.where(beta > 0, a / beta, 0.0)   # s a/beta -> 0 with beta
        dz = -a * (G * prev - G * u * ratio)
        out["dgate"] = dz * _f64(rate) * s * n
        out["drate"] = (dz * s).sum((0, 1))
    return out


def norm_forward(s, weight=None, bias=None, eps=1e-5, rms=False):
    """s: [rows, D] (the sum, already rounded where the operator rounds it).  Returns (y, mean, rstd)."""
    s = _f64(s)
    mean = np.zeros(s.shape[0]) if rms else s.mean(1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(1) + eps)
    y = (s - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean, rstd


def norm_backward(dy, s, weight=None, dresidual=None, eps=1e-5, rms=False):
    """Gradients of a loss whose gradient is dy at y and dresidual at s: (ds, dweight, dbias)."""
    dy, s = _f64(dy), _f64(s)
    _, mean, rstd = norm_forward(s, eps=eps, rms=rms)
    D = s.shape[1]
    z = (s - mean[:, None]) * rstd[:, None]
    w = dy if weight is None else dy * _f64(weight)
    ds = np.empty_like(s)
    for r in range(s.shape[0]):
        # d z_i / d s_j = rstd (delta_ij - 1/D - z_i z_j / D)   (rms: without 1/D)
        m1 = 0.0 if rms else w[r].sum() / D
        ds[r] = rstd[r] * (w[r] - m1 - z[r] * (w[r] @ z[r]) / D)
    if dresidual is not None:
        ds = ds + _f64(dresidual)
    return ds, (dy * z).sum(0), dy.sum(0)
