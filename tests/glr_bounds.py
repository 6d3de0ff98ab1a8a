"""Elementwise error bounds of the gated linear recurrence's kernels, from their arithmetic.

U = 2^-24 is half a step of fp32.  ex2.approx is off by at most 4 U relative, rcp.approx,
sqrt.approx and rsqrt.approx by 2 U, every fp32 operation by U; an exponent's argument e has
absolute error 2 U |e| (the constant log2 e and the product).  Hence
  sigmoid (and its complement)      (8 + 2 |g|) U relative
  z = rate sigmoid                  (9 + 2 |g|) U relative
  1 - a                             z <= 1/8: (17 + 2 |g|) U relative (the polynomial: 5.6 U);
                                    beyond: that of a, absolute
  a                                 z <= 1/8: that of 1 - a, and U; beyond: (z (11 + 2 |g|) + 4) U relative
  beta = sqrt((1 - a)(1 + a))       a d(1 - a) / beta + 4 U beta
The scan joins pieces, so the rounding of a state is counted against the envelope M (the
recurrence of the absolute values), 4 U for a token's own operations and 4 U a for its
factor in every product of decays.  A result in bf16 is rounded once more: 2^-8 relative.
"""
import numpy as np

from oracle import block_oracle as BO

U = 2.0 ** -24


def _pieces(x, gate, rate, ig):
    g = np.abs(gate)
    s, n = BO._sig(gate), BO._sig(-gate)
    a, beta = BO.glr_coefficients(gate, rate)
    if rate is None:
        da = a * (8 + 2 * g) * U
        dbeta = beta * (8 + 2 * g) * U
    else:
        z = rate * s
        m = -np.expm1(-z)
        slow = z <= 0.125 * (1 + 1e-5)
        fast_da = a * (z * (11 + 2 * g) + 4) * U
        dm = np.where(slow, m * (17 + 2 * g) * U, fast_da + U * m)
        da = np.where(slow, dm + U, fast_da)
        with np.errstate(divide="ignore", invalid="ignore"):
            dbeta = np.where(beta > 0, a * dm / beta, 0.0) + 4 * U * beta
    si = np.ones_like(x) if ig is None else BO._sig(ig)
    gi = np.zeros_like(x) if ig is None else np.abs(ig)
    u = np.abs(x * si)
    db = dbeta * u + beta * u * (11 + 2 * gi) * U
    return a, beta, da, dbeta, u, db, s, n, si, gi, g


def _rounded(ref, err, dtype):
    return err + (2.0 ** -8 * (np.abs(ref) + err) if dtype == "bf16" else U * np.abs(ref))


def forward(x, gate, rate, ig, h0, dtype):
    """(y, h_final, bound of y, bound of h_final)"""
    y, hf = BO.glr_forward(x, gate, rate, ig, h0)
    a, beta, da, dbeta, u, db, *_ = _pieces(x, gate, rate, ig)
    M, E = _state_bounds(a, beta, da, u, db, h0)
    eh = E[:, -1] if x.shape[1] else np.zeros_like(hf)
    return y, hf, _rounded(y, E, dtype), eh + U * np.abs(hf)


def _state_bounds(a, beta, da, u, db, h0):
    B, L, D = a.shape
    m = np.zeros((B, D)) if h0 is None else np.abs(h0)
    e = np.zeros((B, D))
    M, E = np.empty_like(a), np.empty_like(a)
    for t in range(L):
        e = a[:, t] * e + (da[:, t] + 4 * U * a[:, t]) * m + db[:, t]
        m = a[:, t] * m + beta[:, t] * u[:, t]
        e = e + 4 * U * m
        M[:, t], E[:, t] = m, e
    return M, E


def backward(x, gate, dy, rate, ig, h0, dhf, dtype):
    """{gradient: (value, bound)}"""
    g = BO.glr_backward(x, gate, dy, rate, ig, h0, dhf)
    a, beta, da, dbeta, u, db, s, n, si, gi, ga = _pieces(x, gate, rate, ig)
    B, L, D = a.shape
    M, E = _state_bounds(a, beta, da, u, db, h0)
    z = np.zeros((B, 1, D))
    Mp = np.concatenate([z if h0 is None else np.abs(h0)[:, None], M[:, :-1]], 1)
    Ep = np.concatenate([z, E[:, :-1]], 1)
    m = np.zeros((B, D)) if dhf is None else np.abs(dhf)
    e = np.zeros((B, D))
    GM, EG = np.empty_like(a), np.empty_like(a)
    for t in range(L - 1, -1, -1):
        GM[:, t] = np.abs(dy[:, t]) + m
        EG[:, t] = e + 4 * U * GM[:, t]
        e = a[:, t] * EG[:, t] + (da[:, t] + 4 * U * a[:, t]) * GM[:, t]
        m = a[:, t] * GM[:, t]
    out = {"dh0": (g["dh0"], e + U * np.abs(g["dh0"]))}
    dx = EG * beta * si + GM * (dbeta * si + beta * si * (13 + 2 * gi) * U)
    out["dx"] = (g["dx"], _rounded(g["dx"], dx, dtype))
    if ig is not None:
        ni = BO._sig(-ig)
        ax = np.abs(x)
        di = EG * beta * ax * si * ni + GM * ax * si * ni * (dbeta + beta * (24 + 4 * gi) * U)
        out["dinput_gate"] = (g["dinput_gate"], _rounded(g["dinput_gate"], di, dtype))
    hp = np.abs(g["prev"])
    if rate is None:
        inner = Ep + u * (9 + 2 * gi) * U + 2 * U * (Mp + u)
        err = EG * (hp + u) * s * n + GM * s * n * (inner + (hp + u) * (20 + 4 * ga) * U)
    else:
        with np.errstate(divide="ignore", invalid="ignore"):
            ib = np.where(beta > 0, 1 / beta, 0.0)
        R = a * ib * u
        dR = (da * ib + a * ib * ib * dbeta) * u + R * (17 + 2 * gi) * U
        inner = Ep + dR + 2 * U * (Mp + R)
        term = a * (hp + R)
        per = s * (EG * term + GM * (a * inner + (hp + R) * (da + a * (26 + 4 * ga) * U)))
        err = rate * n * per
        total = np.abs(GM * s * term)
        out["drate"] = (g["drate"], per.sum((0, 1)) + (L + B + 64) * U * total.sum((0, 1)))
    out["dgate"] = (g["dgate"], _rounded(g["dgate"], err, dtype))
    return out
