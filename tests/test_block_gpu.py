"""The operators together, as a residual block uses them: norm, gated recurrence, residual
addition, next norm; prompt then tokens one by one; and the block's whole backward pass."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from selective_state_space_32_b200 import sscan as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_32_b200 import build
    build.build()
    S.lib()


def rel(a, b):
    a = a.double().cpu().numpy()
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def params(D, seed=0):
    r = np.random.default_rng(seed)
    f = lambda *s: r.standard_normal(s).astype(np.float32)
    return {"w1": 1 + 0.2 * f(D), "b1": 0.2 * f(D), "w2": 1 + 0.2 * f(D), "g": f(D), "i": f(D),
            "rate": np.exp(r.uniform(-4, -0.5, D)).astype(np.float32)}


def block(x, P, h0=None, want_states=False):
    """norm -> (gates from the normed values, per-channel scales) -> recurrence -> residual -> rms norm"""
    n, s, mu, rstd = S.norm_forward(x, P["w1"], P["b1"])
    gate, ig = (n * P["g"]).contiguous(), (n * P["i"]).contiguous()
    y, hf, st = S.glr_forward(n, gate, P["rate"], ig, h0, want_states=want_states)
    out, res, _, rstd2 = S.norm_forward(y, P["w2"], residual=x, rms=True)
    return out, res, hf, (n, s, mu, rstd, gate, ig, st, res, rstd2)


def oracle_block(x, P, h0=None):
    B, L, D = x.shape
    n = BO.norm_forward(x.reshape(-1, D), P["w1"], P["b1"])[0].reshape(B, L, D)
    y, hf = BO.glr_forward(n, n * P["g"], P["rate"], n * P["i"], h0)
    res = x + y
    out = BO.norm_forward(res.reshape(-1, D), P["w2"], None, rms=True)[0].reshape(B, L, D)
    return out, res, hf, n, y


@pytest.mark.parametrize("shape", [(2, 300, 136), (1, 1500, 65), (3, 9, 512)])
def test_prompt_and_tokens(shape):
    """A prompt in one call and the rest token by token give the whole sequence's outputs (fp32: a chain of
    three operators, each within ~1e-6 relative; 1e-5 is the repository's fp32 tolerance)."""
    B, L, D = shape
    P = params(D)
    C = {k: torch.from_numpy(v).cuda() for k, v in P.items()}
    x = np.random.default_rng(1).standard_normal((B, L, D)).astype(np.float32)
    xc = torch.from_numpy(x).cuda()
    want, wres, whf, _, _ = oracle_block(x.astype(np.float64), {k: v.astype(np.float64) for k, v in P.items()})
    out, res, hf, _ = block(xc, C)
    assert rel(out, want) < 1e-5 and rel(res, wres) < 1e-5 and rel(hf, whf) < 1e-5
    cut = L - 6
    h, outs = torch.zeros(B, D, device="cuda"), []
    o, _, h, _ = block(xc[:, :cut].clone(), C, h)
    outs.append(o)
    for t in range(cut, L):
        o, _, h, _ = block(xc[:, t:t + 1].clone(), C, h)   # of its own: a view of an odd row would not be aligned
        outs.append(o)
    assert rel(torch.cat(outs, 1), want) < 1e-5 and rel(h, whf) < 1e-5


def test_bf16_block_with_the_residual_stream_in_fp32():
    B, L, D = 2, 500, 264
    P = params(D, 2)
    C = {k: torch.from_numpy(v).cuda() for k, v in P.items()}
    x = torch.randn(B, L, D, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()
    res = torch.randn(B, L, D, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    n, s, _, _ = S.norm_forward(x, C["w1"], C["b1"], residual=res)
    assert n.dtype == torch.bfloat16 and s.dtype == torch.float32
    gate = (n.float() * C["g"]).bfloat16()
    y, hf, _ = S.glr_forward(n, gate, C["rate"])
    out, s2, _, _ = S.norm_forward(y, C["w2"], residual=s, rms=True)
    n_, g_ = n.double().cpu().numpy(), gate.double().cpu().numpy()
    yr, hr = BO.glr_forward(n_, g_, P["rate"])
    assert rel(y, yr) < 5e-3 and rel(hf, hr) < 1e-5
    want = BO.norm_forward((s.double().cpu().numpy() + yr).reshape(-1, D), P["w2"], rms=True)[0].reshape(B, L, D)
    assert rel(out, want) < 5e-3


@pytest.mark.parametrize("shape", [(2, 260, 72), (1, 1100, 65)])
def test_backward_through_the_block(shape):
    """The block's gradients, composed from the operators' backward passes, against the oracle's
    composed the same way (which differences pin operator by operator)."""
    B, L, D = shape
    P = params(D, 3)
    C = {k: torch.from_numpy(v).cuda() for k, v in P.items()}
    r = np.random.default_rng(7)
    x = r.standard_normal((B, L, D)).astype(np.float32)
    dout = r.standard_normal((B, L, D)).astype(np.float32)
    xc, do = torch.from_numpy(x).cuda(), torch.from_numpy(dout).cuda()
    out, res, hf, (n, s, mu, rstd, gate, ig, st, res, rstd2) = block(xc, C, want_states=True)
    b2 = S.norm_backward(do, res, None, rstd2, C["w2"], rms=True)
    g = S.glr_backward(n, gate, b2["dx"], st, C["rate"], ig)
    dn = g["dx"] + g["dgate"] * C["g"] + g["dinput_gate"] * C["i"]
    b1 = S.norm_backward(dn, s, mu, rstd, C["w1"], dresidual=b2["dresidual"], want_dbias=True)

    Q = {k: v.astype(np.float64) for k, v in P.items()}
    xd = x.astype(np.float64)
    _, wres, _, wn, wy = oracle_block(xd, Q)
    d2, dw2, _ = BO.norm_backward(dout.reshape(-1, D), wres.reshape(-1, D), Q["w2"], rms=True)
    d2 = d2.reshape(B, L, D)
    wg = BO.glr_backward(wn, wn * Q["g"], d2, Q["rate"], wn * Q["i"])
    wdn = wg["dx"] + wg["dgate"] * Q["g"] + wg["dinput_gate"] * Q["i"]
    d1, dw1, db1 = BO.norm_backward(wdn.reshape(-1, D), xd.reshape(-1, D), Q["w1"], d2.reshape(-1, D))
    for got, want in ((b1["dx"], d1.reshape(B, L, D)), (b2["dweight"], dw2), (b1["dweight"], dw1), (b1["dbias"], db1),
                      (g["drate"], wg["drate"]), (g["dh0"], wg["dh0"])):
        assert rel(got, want) < 1e-5
