"""The oracle of the gated linear recurrence and the layer norm: its forward functions
against independent forms, its gradients against central differences (CPU, fp64)."""
import numpy as np
import pytest

from oracle import block_oracle as BO
from oracle import oracle as O


def _inputs(B, L, D, ig, decay, state, seed=1):
    r = np.random.default_rng(seed)
    return {"x": r.standard_normal((B, L, D)), "gate": r.standard_normal((B, L, D)) + 1.0,
            "rate": np.exp(r.uniform(-3, 0, D)) if decay else None,
            "input_gate": r.standard_normal((B, L, D)) if ig else None,
            "h0": r.standard_normal((B, D)) if state else None}


def test_without_a_rate_it_is_the_scan_of_the_gru_identity():
    """N = 1, A = -1, B = C = 1, exact ZOH, delta = softplus(v): h = (1 - sigmoid(v)) h + sigmoid(v) u,
    which is the recurrence with gate = -v."""
    r = np.random.default_rng(0)
    B, L, D = 2, 37, 5
    v, u, h0 = (r.standard_normal(s).astype(np.float32) for s in ((B, L, D), (B, L, D), (B, D, 1)))
    one = np.ones((B, L, 1), np.float32)
    y, hf = O.forward(u, v, -np.ones((D, 1), np.float32), one, one, h0, True, softplus=True)
    yo, ho = BO.glr_forward(u, -v, h0=h0[:, :, 0])
    assert np.allclose(yo, y, rtol=1e-12, atol=1e-13) and np.allclose(ho, hf[:, :, 0], rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("decay", [False, True])
def test_unrolled_sum(decay):
    """y_t = (prod_{k<=t} a_k) h0 + sum_j (prod_{j<k<=t} a_k) beta_j u_j"""
    d = _inputs(2, 9, 3, True, decay, True)
    a, beta = BO.glr_coefficients(d["gate"], d["rate"])
    u = d["x"] / (1 + np.exp(-d["input_gate"]))
    y, _ = BO.glr_forward(**d)
    for t in range(9):
        want = np.prod(a[:, :t + 1], axis=1) * d["h0"]
        for j in range(t + 1):
            want = want + np.prod(a[:, j + 1:t + 1], axis=1) * beta[:, j] * u[:, j]
        assert np.allclose(y[:, t], want, rtol=1e-12)
    if decay:
        assert np.allclose(a ** 2 + beta ** 2, 1.0, rtol=1e-12)


@pytest.mark.parametrize("decay", [False, True])
@pytest.mark.parametrize("ig", [False, True])
def test_recurrence_gradients_by_differences(decay, ig):
    B, L, D = 2, 6, 3
    d = _inputs(B, L, D, ig, decay, True, seed=3)
    r = np.random.default_rng(4)
    dy, dhf = r.standard_normal((B, L, D)), r.standard_normal((B, D))

    def loss(q):
        y, hf = BO.glr_forward(**q)
        return (y * dy).sum() + (hf * dhf).sum()
    g = BO.glr_backward(d["x"], d["gate"], dy, d["rate"], d["input_gate"], d["h0"], dhf)
    for name, grad in (("x", "dx"), ("gate", "dgate"), ("input_gate", "dinput_gate"), ("rate", "drate"), ("h0", "dh0")):
        if d[name] is None:
            assert g[grad] is None
            continue
        num = np.empty_like(d[name])
        for i in np.ndindex(*d[name].shape):
            v = []
            for e in (1e-6, -1e-6):
                q = dict(d, **{name: d[name].copy()})
                q[name][i] += e
                v.append(loss(q))
            num[i] = (v[0] - v[1]) / 2e-6
        # differences of fp64 losses of size ~10: 1e-15 * 10 / 1e-6, and the cubic term ~1e-12
        assert np.allclose(num, g[grad], atol=1e-7, rtol=1e-7), name


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_by_differences(rms):
    r = np.random.default_rng(5)
    s, w, b = r.standard_normal((3, 7)) + 0.5, r.standard_normal(7), r.standard_normal(7)
    dy, dr = r.standard_normal((3, 7)), r.standard_normal((3, 7))

    def loss(s, w, b):
        return (BO.norm_forward(s, w, b, rms=rms)[0] * dy).sum() + (s * dr).sum()
    got = BO.norm_backward(dy, s, w, dr, rms=rms)
    for k, (p, g) in enumerate(zip((s, w, b), got)):
        num = np.empty_like(p)
        for i in np.ndindex(*p.shape):
            v = []
            for e in (1e-6, -1e-6):
                q = [s.copy(), w.copy(), b.copy()]
                q[k][i] += e
                v.append(loss(*q))
            num[i] = (v[0] - v[1]) / 2e-6
        assert np.allclose(num, g, atol=1e-7, rtol=1e-7), k


def test_norm_statistics():
    r = np.random.default_rng(6)
    s = r.standard_normal((4, 33)) * 3 + 100
    y, mean, rstd = BO.norm_forward(s, eps=0.0)
    assert np.allclose(y.mean(1), 0, atol=1e-12) and np.allclose((y ** 2).mean(1), 1)
    y, mean, rstd = BO.norm_forward(s, eps=0.0, rms=True)
    assert np.all(mean == 0) and np.allclose((y ** 2).mean(1), 1) and np.allclose(y * np.sqrt((s ** 2).mean(1))[:, None], s)
