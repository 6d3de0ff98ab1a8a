"""The rate's gradient, a sum over a whole walk: checks that a lost warp or block cannot pass.

drate = -sum over rows and tokens of G_t s_t a_t (h_{t-1} - (a_t / beta_t) u_t).  With x > 0, dy > 0 and a
large state in front of them the states and G are positive and nearly every term has one sign, so that
each warp's share shows: with 128 warps on a walk a lost one takes 1/128 of the sum.  The bound counts the
additions that a term meets: the tokens of a thread, at most 8 warps, the blocks' rows in steps of 256,
the two trees of 3 and 5.  With x and dy of both signs the sum cancels down to the root of the number
of terms, and a lost warp shows in the relative L2 norm over the channels (1e-5: the
repository's fp32 tolerance)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from selective_state_space_32_b200 import sscan as S
from tests import glr_bounds as GB
from tests.test_glr_gpu import cuda, host, make

RUN = 8   # tokens of a warp's run in the backward pass
# B, L, D, dtype, and the warps that share a walk (blocks of a cluster times warps of a block)
CASES = [(1, 40000, 64, "bf16", 128), (1, 9000, 96, "f32", 128), (2, 3000, 1024, "bf16", 64), (8, 600, 1536, "bf16", 8),
         (3, 300, 512, "f32", 64), (1, 20000, 40, "f32", 128), (2, 2000, 101, "bf16", 64), (70, 17, 96, "f32", 4)]


def inputs(B, L, D, dtype, positive):
    d = make(B, L, D, dtype, True, True, False, seed=21)
    if positive:
        d["x"], d["dy"] = d["x"].abs() + 0.5, d["dy"].abs() + 0.5
    d["h0"] = torch.full((B, D), 40.0) if positive else None
    d["dh_final"] = None
    return d


def terms(v):
    g = BO.glr_backward(v["x"], v["gate"], v["dy"], v["rate"], v["input_gate"], v["h0"])
    a, beta = BO.glr_coefficients(v["gate"], v["rate"])
    u = v["x"] * BO._sig(v["input_gate"])
    return -g["G"] * BO._sig(v["gate"]) * a * (g["prev"] - a / beta * u), g["drate"]


def bound(v, dtype, L, B, warps):
    """The terms' own errors (glr_bounds.py, without its allowance for the sum) and the sum's."""
    t, _ = terms(v)
    full = GB.backward(v["x"], v["gate"], v["dy"], v["rate"], v["input_gate"], v["h0"], None, dtype)["drate"][1]
    a, beta = BO.glr_coefficients(v["gate"], v["rate"])
    u = v["x"] * BO._sig(v["input_gate"])
    g = BO.glr_backward(v["x"], v["gate"], v["dy"], v["rate"], v["input_gate"], v["h0"])   # x, dy, h0 > 0
    size = (g["G"] * BO._sig(v["gate"]) * a * (g["prev"] + a / beta * u)).sum((0, 1))
    own = full - (L + B + 64) * GB.U * size
    assert (own >= 0).all()
    steps = -(-(-(-L // RUN)) // warps)
    depth = steps * RUN + 8 + -(-B * min(16, warps) // 256) + 3 + 5
    return own + depth * GB.U * size


def shares(t, warps):
    """The sum of each warp's terms [warps, D]: runs in turn from the last one."""
    B, L, D = t.shape
    runs = -(-L // RUN)
    p = np.zeros((B, runs * RUN, D))
    p[:, :L] = t
    per_run = p.reshape(B, runs, RUN, D).sum((0, 2))[::-1]
    return np.stack([per_run[w::warps].sum(0) for w in range(min(warps, runs))])


# the walks whose warps have many terms each
@pytest.mark.parametrize("B,L,D,dtype,warps", CASES[:4] + CASES[5:6])
def test_a_lost_warp_would_show(B, L, D, dtype, warps):
    """The checks below against a reference that lacks one warp's terms: each of them fails."""
    v = host(inputs(B, L, D, dtype, True))
    t, ref = terms(v)
    b = bound(v, dtype, L, B, warps)
    assert np.allclose(t.sum((0, 1)), ref, rtol=1e-9)
    lost = np.abs(shares(t, warps))
    assert (lost > 2 * b).all(), (lost / b).min()
    t, ref = terms(host(inputs(B, L, D, dtype, False)))
    lost = np.linalg.norm(shares(t, warps), axis=1) / np.linalg.norm(ref)
    assert (lost > 1e-3).all()


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_32_b200 import build
    build.build()
    S.lib()


def drate(c):
    _, _, st = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], c["h0"], want_states=True)
    return S.glr_backward(c["x"], c["gate"], c["dy"], st, c["rate"], c["input_gate"])["drate"].double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,D,dtype,warps", CASES)
def test_terms_of_one_sign(device, B, L, D, dtype, warps):
    d = inputs(B, L, D, dtype, True)
    v = host(d)
    _, ref = terms(v)
    over = np.abs(drate(cuda(d)) - ref) / bound(v, dtype, L, B, warps)
    assert over.max() <= 1.0, (over.max(), int(over.argmax()))


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,D,dtype,warps", CASES)
def test_terms_of_both_signs(device, B, L, D, dtype, warps):
    d = inputs(B, L, D, dtype, False)
    _, ref = terms(host(d))
    got = drate(cuda(d))
    assert np.linalg.norm(got - ref) <= 1e-5 * np.linalg.norm(ref)


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,D,dtype,warps", CASES)
def test_one_run_at_a_time(device, B, L, D, dtype, warps):
    """dy at a single token that nothing precedes but zeros (x = 0 before it), in one run after another:
    drate is that token's term and its neighbours' alone, whichever warp and block it falls to."""
    r = np.random.default_rng(3)
    d = inputs(B, L, D, dtype, True)
    runs = -(-L // RUN)
    for q in sorted({0, 1, runs - 1, *r.integers(0, runs, 6).tolist()}):
        at = min(q * RUN + int(r.integers(0, RUN)), L - 1)
        e = {k: None if w is None else w.clone() for k, w in d.items()}
        e["h0"] = None
        e["x"][:, :max(at - 1, 0)] = 0
        e["dy"][:, :at], e["dy"][:, at + 1:] = 0, 0
        v = host(e)
        lo = max(at - 1, 0)
        part = {k: (w if w is None or k == "rate" else w[:, lo:at + 1]) for k, w in v.items() if k not in ("dh_final", "h0")}
        ref, b = GB.backward(part["x"], part["gate"], part["dy"], part["rate"], part["input_gate"], None, None, dtype)["drate"]
        got = drate(cuda(e))
        assert (np.abs(got - ref) <= b).all() and (np.abs(ref) > 10 * b).mean() > 0.9, at
