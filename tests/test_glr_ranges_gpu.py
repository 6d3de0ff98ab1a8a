"""GPU tests of the gated linear recurrence at the ends of its inputs' ranges: large rates, closed
input gates.  Against the fp64 oracle, elementwise, with the bounds of glr_bounds.py."""
import numpy as np
import pytest
import torch

from selective_state_space_32_b200 import sscan as S
from tests import glr_bounds as GB
from tests.test_glr_gpu import DT, close, cuda, host, make

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_32_b200 import build
    build.build()
    S.lib()


def compare(d, dtype, ytol=0.0, gtol=0.0):
    v, c = host(d), cuda(d)
    y, hf, st = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], c["h0"], want_states=True)
    g = S.glr_backward(c["x"], c["gate"], c["dy"], st, c["rate"], c["input_gate"], c["dh_final"])
    yr, hr, by, bh = GB.forward(v["x"], v["gate"], v["rate"], v["input_gate"], v["h0"], dtype)
    want = GB.backward(v["x"], v["gate"], v["dy"], v["rate"], v["input_gate"], v["h0"], v["dh_final"], dtype)
    close(y, yr, by + ytol, "y")
    close(hf, hr, bh + ytol, "h_final")
    for k, (ref, bound) in want.items():
        close(g[k], ref, bound + gtol, k)
    return v, y, g


# step kernel, one block, a walk of several blocks; rows of 16-byte vectors and others
SHAPES = [(2, 3, 72), (2, 300, 72), (2, 300, 71), (1, 2000, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ig", [False, True])
@pytest.mark.parametrize("B,L,D", SHAPES)
@pytest.mark.parametrize("lo,hi", [(81.0, 1e4), (1e4, 2.0 ** 21)])
def test_large_rates_with_closed_gates(B, L, D, dtype, ig, lo, hi):
    """exp(-rate sigmoid(gate)) where the rate is large and the gate is near the point that makes their
    product 1, or open.  Decays below 2^-126 are up to 2^-125.5: with |x|, |dy|, |h0| < 6, and so
    |h|, |G|, |u / beta| < 1e4, that is off by at most 2^-126 (1 + rate) 1e10."""
    d = make(B, L, D, dtype, True, ig, True, seed=5)
    r = np.random.default_rng(11)
    rate = np.exp(r.uniform(np.log(lo), np.log(hi), D)).astype(np.float32)
    gate = np.where(r.random((B, L, D)) < 0.1, r.uniform(-1, 3, (B, L, D)), 1.5 * r.standard_normal((B, L, D)) - np.log(rate))
    d["rate"] = torch.from_numpy(rate)
    d["gate"] = torch.from_numpy(gate.astype(np.float32)).to(d["gate"].dtype)
    v, y, g = compare(d, dtype, TINY * 1e10, TINY * (1 + hi) * 1e10)
    a = np.exp(-v["rate"] / (1 + np.exp(-v["gate"])))
    assert (a < 0.01).mean() > 0.1 and (a > 0.5).mean() > 0.1   # both are met


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [3, 300])
@pytest.mark.parametrize("rate", [2.0 ** 21, 1e9, 3e38, float("inf")])
def test_the_largest_rates_forget_at_every_open_gate(rate, L, dtype):
    """a = 0 and beta = 1 wherever the gate is above -9.5 (rate times sigmoid at least 157), the state
    held at -infinity; no gradient through the gate or the rate (but for 2^-126 of the factors' size)."""
    d = cuda(make(2, L, 72, dtype, True, True, True))
    d["rate"].fill_(rate)
    d["gate"].mul_(3).clamp_(min=-9.5)
    d["gate"][:, ::3] = -float("inf")
    y, hf, st = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"], want_states=True)
    g = S.glr_backward(d["x"], d["gate"], d["dy"], st, d["rate"], d["input_gate"], d["dh_final"])
    u = d["x"].double() * torch.sigmoid(d["input_gate"].double())
    want, h = torch.empty_like(u), d["h0"].double()
    for t in range(L):
        h = h if t % 3 == 0 else u[:, t]
        want[:, t] = h
    half = torch.finfo(d["x"].dtype).eps / 2
    # the input gate's sigmoid (8 + 2 |ig|) U, four more operations, and the rounding
    tol = (half + (12 + 2 * d["input_gate"].double().abs().max()) * 2.0 ** -24) * u.abs().max() + 1e2 * TINY
    assert (y.double() - want).abs().max() <= (2.0 ** -24 + half) * d["h0"].abs().max() + tol
    assert all(torch.isfinite(q).all() for q in g.values())
    # backward a closed gate is 2^-126 and a rate at most 2^21: z = 2^-105, beta = sqrt(2 z) = 2^-52,
    # dgate G u sqrt(z / 2), drate that over the rate, summed; |G| < 20, |u| < 6
    assert g["dx"][:, ::3].abs().max() <= 20 * 2.0 ** -52
    assert g["dgate"].abs().max() <= 120 * 2.0 ** -53 and g["drate"].abs().max() <= 2 * L * 120 * 2.0 ** -74


def test_a_rate_of_nan_is_nan_in_its_channel_only():
    d = cuda(make(2, 40, 72, "f32", True, True, True))
    want = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"])[0]
    d["rate"][5] = float("nan")
    y = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"])[0]
    keep = [i for i in range(72) if i != 5]
    assert torch.isnan(y[..., 5]).all() and torch.equal(y[..., keep], want[..., keep])


@pytest.mark.parametrize("decay", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", SHAPES)
def test_input_gates_far_closed(B, L, D, dtype, decay):
    """Input gates from -30 to -80 (sigmoids from 1e-13 to 2e-35) let their share through: a state that
    only such gates feed has the oracle's relative digits.  fp32's smallest normal number times the
    tokens is left to operands that become subnormal."""
    d = make(B, L, D, dtype, decay, True, False, seed=9)
    r = np.random.default_rng(12)
    lo = np.linspace(-78, -32, D)   # a channel's gates are near each other, so that none hides the others
    d["input_gate"] = torch.from_numpy((lo + r.uniform(-2, 2, (B, L, D))).astype(np.float32)).to(DT[dtype])
    v, y, g = compare(d, dtype, L * TINY, L * TINY)
    assert (y != 0).float().mean() > 0.99


@pytest.mark.parametrize("L", [2, 40])
def test_an_input_gate_of_nan_is_nan_and_one_of_minus_infinity_nothing(L):
    d = cuda(make(1, L, 72, "f32", True, True, True))
    d["input_gate"][:, :, 3] = -float("inf")
    d["input_gate"][0, 1, 9] = float("nan")
    y = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"])[0]
    none = S.glr_forward(d["x"] * 0, d["gate"], d["rate"], d["input_gate"], d["h0"])[0]
    assert (y[..., 3] - none[..., 3]).abs().max() <= 1e-30 and torch.isfinite(y[:, 0]).all()
    assert torch.isnan(y[0, 1:, 9]).all()


@pytest.mark.parametrize("decay", [False, True])
@pytest.mark.parametrize("ig", [False, True])
@pytest.mark.parametrize("L", [1, 3, 20, 400])
def test_inputs_near_the_largest_number(L, ig, decay):
    """x close to fp32's largest value is not taken past it on its way to the state."""
    d = make(1, L, 72, "f32", decay, ig, False, seed=3)
    r = np.random.default_rng(4)
    at = torch.from_numpy(r.integers(0, L, 72))
    d["x"][0, at, torch.arange(72)] = torch.from_numpy((r.choice([-1, 1], 72) * r.uniform(2e38, 3.4e38, 72)).astype(np.float32))
    if ig:
        d["input_gate"][:, :, ::2] = 30.0
    v, c = host(d), cuda(d)
    y, hf, _ = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], c["h0"])
    yr, hr, by, bh = GB.forward(v["x"], v["gate"], v["rate"], v["input_gate"], v["h0"], "f32")
    close(y, yr, by, "y")
    close(hf, hr, bh, "h_final")
