"""GPU tests of the gated linear recurrence against the fp64 oracle, elementwise, with the
bounds of glr_bounds.py (derived from the kernels' arithmetic, no free factor)."""
import numpy as np
import pytest
import torch

from selective_state_space_32_b200 import sscan as S
from tests import glr_bounds as GB

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_32_b200 import build
    build.build()
    S.lib()


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(B, L, D, dtype, decay, ig, state, seed=0):
    r = np.random.default_rng(seed + 7919 * L + D)
    t = lambda *s, m=0.0: torch.from_numpy((r.standard_normal(s) + m).astype(np.float32)).to(DT[dtype])
    f = lambda v: torch.from_numpy(np.asarray(v, np.float32))
    d = {"x": t(B, L, D), "gate": t(B, L, D, m=0.0 if decay else 1.5),
         "rate": f(np.exp(r.uniform(np.log(0.008), np.log(0.8), D))) if decay else None,
         "input_gate": t(B, L, D) if ig else None, "h0": f(r.standard_normal((B, D))) if state else None,
         "dy": t(B, L, D), "dh_final": f(r.standard_normal((B, D))) if state else None}
    return d


def host(d):
    return {k: None if v is None else v.double().numpy() for k, v in d.items()}


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def num(t):
    return t.double().cpu().numpy()


def close(got, ref, bound, what):
    got = num(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not got.size:
        return
    over = np.abs(got - ref) / np.maximum(bound, 1e-300)
    over[(got == ref)] = 0.0
    i = np.unravel_index(np.nanargmax(np.where(np.isnan(over), np.inf, over)), over.shape)
    assert over[i] <= 1.0, f"{what}{i}: got {got[i]!r}, want {ref[i]!r}, bound {bound[i]!r}"


def check(B, L, D, dtype, decay, ig, state, seed=0):
    d = make(B, L, D, dtype, decay, ig, state, seed)
    v, c = host(d), cuda(d)
    y, hf, states = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], c["h0"], want_states=True)
    yr, hr, by, bh = GB.forward(v["x"], v["gate"], v["rate"], v["input_gate"], v["h0"], dtype)
    close(y, yr, by, "y")
    close(hf, hr, bh, "h_final")
    y2, hf2, none = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], c["h0"])
    assert none is None and torch.equal(y, y2) and torch.equal(hf, hf2)   # saving states changes nothing
    g = S.glr_backward(c["x"], c["gate"], c["dy"], states, c["rate"], c["input_gate"], c["dh_final"])
    want = GB.backward(v["x"], v["gate"], v["dy"], v["rate"], v["input_gate"], v["h0"], v["dh_final"], dtype)
    assert (g["drate"] is None) == (not decay) and (g["dinput_gate"] is None) == (not ig)
    for k, (ref, bound) in want.items():
        close(g[k], ref, bound, k)
    return c, y, hf, states, g


FORMS = [(dec, ig) for dec in (False, True) for ig in (False, True)]
LENGTHS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 63, 64, 65, 127, 129, 511, 512, 513, 777, 1025, 2049]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", LENGTHS)
def test_lengths(L, dtype):
    for k, (decay, ig) in enumerate(FORMS):
        check(2, L, [64, 72, 70, 65][(L + k) % 4], dtype, decay, ig, (L + k) % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 7, 8, 24, 31, 32, 33, 63, 100, 128, 136, 250, 515])
def test_widths(D, dtype):
    for decay, ig in FORMS:
        check(3, 70, D, dtype, decay, ig, D % 2 == 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_long_sequence(dtype):
    check(1, 20000, 40, dtype, True, True, True)
    check(1, 9001, 8, dtype, False, False, False)


@pytest.mark.parametrize("B,L,D", [(300, 1, 64), (64, 3, 515), (40, 33, 264), (5, 300, 1032)])
def test_many_rows(B, L, D):
    check(B, L, D, "f32", True, True, True)
    check(B, L, D, "bf16", False, True, True)


@pytest.mark.parametrize("B,L,D,dtype", [
    (1, 40000, 64, "bf16"),      # one chain: clusters of 16 blocks of 8 warps
    (1, 9000, 96, "f32"),        # three chains
    (2, 3000, 1024, "bf16"),     # 32 chains: clusters of 8
    (8, 600, 1536, "bf16"),      # 192 chains: clusters of 2
    (3, 300, 4096, "f32"),       # 384 chains: one block each, of 4 warps or of 8
    (70, 17, 8000, "f32"),       # 17500 chains: one warp each
    (3, 1000, 515, "bf16"),      # rows that are not a multiple of 16 bytes
])
def test_every_spread_of_the_walk(B, L, D, dtype):
    check(B, L, D, dtype, True, L % 2 == 0, True)


def test_offsets_past_32_bits():
    """2.2e9 values: the end of the sequence against a call on the end alone, from the state before it
    (fp32: y holds the states), both within 1e-5 relative, the repository's fp32 tolerance."""
    B, L, D, tail = 1, 1_060_000, 2056, 3000
    gen = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    x, gate, dy = new(B, L, D), new(B, L, D), new(B, L, D)
    rate = torch.rand(D, device="cuda", generator=gen) * 0.5 + 0.01
    y, hf, st = S.glr_forward(x, gate, rate, want_states=True)
    g = S.glr_backward(x, gate, dy, st, rate)
    cut = L - tail
    part = [t[:, cut:].clone() for t in (x, gate, dy)]
    y2, hf2, st2 = S.glr_forward(part[0], part[1], rate, h0=y[:, cut - 1].contiguous(), want_states=True)
    g2 = S.glr_backward(part[0], part[1], part[2], st2, rate)
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())
    assert rel(y[:, cut:], y2) < 1e-5 and rel(hf, hf2) < 1e-5
    assert rel(g["dx"][:, cut:], g2["dx"]) < 1e-5 and rel(g["dgate"][:, cut:], g2["dgate"]) < 1e-5
    # the first tokens' outputs do not depend on what follows
    assert rel(y[:, :tail], S.glr_forward(x[:, :tail].clone(), gate[:, :tail].clone(), rate)[0]) < 1e-5


def test_rates_above_80_act_as_80():
    d = cuda(make(2, 300, 72, "f32", True, True, True))
    d["rate"][::3] = 80.0
    args = lambda r: (d["x"], d["gate"], r, d["input_gate"], d["h0"])
    more = d["rate"].clone()
    more[::3] = torch.tensor([1e3, float("inf"), 81.0, 1e30] * 6, device="cuda")
    y, hf, st = S.glr_forward(*args(d["rate"]), want_states=True)
    y2, hf2, st2 = S.glr_forward(*args(more), want_states=True)
    assert torch.equal(y, y2) and torch.equal(hf, hf2) and torch.isfinite(y).all()
    a = S.glr_backward(d["x"], d["gate"], d["dy"], st, d["rate"], d["input_gate"])
    b = S.glr_backward(d["x"], d["gate"], d["dy"], st2, more, d["input_gate"])
    assert all(torch.equal(a[k], b[k]) and torch.isfinite(a[k]).all() for k in a)


def test_empty_sequence():
    d = cuda(make(2, 0, 24, "bf16", True, True, True))
    y, hf, st = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"], want_states=True)
    assert y.shape == (2, 0, 24) and torch.equal(hf, d["h0"]) and st.numel() == 0
    assert torch.equal(S.glr_forward(d["x"], d["gate"])[1], torch.zeros(2, 24, device="cuda"))
    g = S.glr_backward(d["x"], d["gate"], d["dy"], st, d["rate"], d["input_gate"], d["dh_final"])
    assert torch.equal(g["dh0"], d["dh_final"]) and not g["drate"].any() and g["dx"].shape == (2, 0, 24)


@pytest.mark.parametrize("L", [1, 3, 100, 700])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_state_in_place_and_in_pieces(L, dtype):
    """h_final over h0, and a sequence cut in two calls, give the one call's results within the bounds."""
    d = make(2, L, 72, dtype, True, True, True)
    v, c = host(d), cuda(d)
    yr, hr, by, bh = GB.forward(v["x"], v["gate"], v["rate"], v["input_gate"], v["h0"], dtype)
    h = c["h0"].clone()
    y, hf, _ = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], h, h_final=h)
    assert hf is h
    close(y, yr, by, "y")
    close(h, hr, bh, "h")
    cut = L // 2
    h, ys = c["h0"].clone(), []
    for a, b in ((0, cut), (cut, L)):
        p = {k: c[k][:, a:b].contiguous() for k in ("x", "gate", "input_gate")}
        ys.append(S.glr_forward(p["x"], p["gate"], c["rate"], p["input_gate"], h, h_final=h)[0])
    close(torch.cat(ys, 1), yr, by, "y in pieces")
    close(h, hr, bh, "h in pieces")


@pytest.mark.parametrize("B,L,D,dtype", [(1, 17, 64, "bf16"), (1, 200, 64, "bf16"), (1, 4100, 40, "f32"), (3, 900, 101, "bf16"),
                                         (2, 3000, 96, "f32")])
def test_state_in_place_across_blocks(B, L, D, dtype):
    """The blocks of a walk all start from h0, also where the walk's end overwrites it."""
    c = cuda(make(B, L, D, dtype, True, True, True, seed=L))
    y, hf, _ = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], c["h0"])
    for _ in range(50):
        h = c["h0"].clone()
        yi, hi, _ = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], h, h_final=h)
        assert hi is h and torch.equal(yi, y) and torch.equal(h, hf)


def test_token_by_token_equals_the_sequence():
    d = make(3, 40, 136, "f32", True, False, True)
    v, c = host(d), cuda(d)
    yr, hr, by, bh = GB.forward(v["x"], v["gate"], v["rate"], None, v["h0"], "f32")
    h, ys = c["h0"].clone(), []
    for t in range(40):
        ys.append(S.glr_forward(c["x"][:, t:t + 1].contiguous(), c["gate"][:, t:t + 1].contiguous(), c["rate"], h0=h,
                                h_final=h)[0])
    close(torch.cat(ys, 1), yr, by, "y")
    close(h, hr, bh, "h")


@pytest.mark.parametrize("L", [1, 30, 600])
@pytest.mark.parametrize("decay", [False, True])
def test_gates_at_infinity_hold_and_replace(L, decay):
    """gate = -inf: without a rate the state is replaced by u, with one it is held exactly (beta = 0);
    gate = +inf: without a rate it is held, with one it decays by exp(-rate)."""
    d = make(2, L, 72, "f32", decay, True, True)
    r = np.random.default_rng(1)
    for val in (-np.inf, np.inf):
        d["gate"][torch.from_numpy(r.random(d["gate"].shape) < 0.3)] = float(val)
    d["gate"][0, :, 5] = -np.inf
    d["input_gate"][torch.from_numpy(r.random(d["gate"].shape) < 0.1)] = -np.inf
    v, c = host(d), cuda(d)
    y, hf, st = S.glr_forward(c["x"], c["gate"], c["rate"], c["input_gate"], c["h0"], want_states=True)
    fin = lambda q: None if q is None else np.clip(q, -80, 80)   # sigmoid(+-80): 1 and 2e-35
    yr, hr, by, bh = GB.forward(v["x"], fin(v["gate"]), v["rate"], fin(v["input_gate"]), v["h0"], "f32")
    close(y, yr, by + 1e-15, "y")
    if decay:
        assert torch.equal(y[0, :, 5], c["h0"][0, 5].expand(L))
    g = S.glr_backward(c["x"], c["gate"], c["dy"], st, c["rate"], c["input_gate"], c["dh_final"])
    want = GB.backward(v["x"], fin(v["gate"]), v["dy"], v["rate"], fin(v["input_gate"]), v["h0"], v["dh_final"], "f32")
    for k, (ref, bound) in want.items():
        # sigmoid(80)'s complement 1.8e-35 stands for 0: beta 1e-17, 1/beta 1e17 times s = 1e-35
        close(g[k], ref, bound + 1e-14 * (1 + np.abs(ref)), k)


def test_very_closed_gates_have_finite_gradients():
    """rate * sigmoid(gate) below fp32's smallest normal number: beta = 0, and the products with 1/beta vanish."""
    d = cuda(make(1, 50, 64, "f32", True, True, True))
    d["gate"].fill_(-86.0)
    d["gate"][:, ::3] = -200.0
    y, hf, st = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"], want_states=True)
    assert (y - d["h0"][:, None]).abs().max() < 1e-14
    g = S.glr_backward(d["x"], d["gate"], d["dy"], st, d["rate"], d["input_gate"], d["dh_final"])
    for k, q in g.items():
        assert torch.isfinite(q).all(), k
    assert g["dgate"].abs().max() < 1e-14 and g["drate"].abs().max() < 1e-12


@pytest.mark.parametrize("L", [5, 900])
def test_a_non_finite_input_stays_in_its_channel_and_after_its_token(L):
    d = cuda(make(2, L, 136, "f32", True, True, True))
    ref = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"])[0]
    for name, val, (b, t, ch) in (("x", float("nan"), (1, L // 2, 7)), ("x", float("inf"), (0, L // 3, 130)),
                                  ("gate", float("nan"), (0, L - 1, 0))):
        q = {k: None if w is None else w.clone() for k, w in d.items()}
        q[name][b, t, ch] = val
        y, hf, _ = S.glr_forward(q["x"], q["gate"], q["rate"], q["input_gate"], q["h0"])
        mask = torch.zeros_like(y, dtype=torch.bool)
        mask[b, t:, ch] = True
        assert torch.equal(y[~mask], ref[~mask])
        assert not torch.isfinite(y[mask]).any()
        assert not torch.isfinite(hf[b, ch])


def test_the_same_call_gives_the_same_bits_and_touches_nothing_else():
    B, L, D = 2, 1100, 200
    d = cuda(make(B, L, D, "bf16", True, True, True))
    ny, ns = B * L * D, S.new_glr_states(B, L, D).numel()
    first = None
    for _ in range(3):
        big = torch.full((ny + 1024,), 7.0, dtype=torch.bfloat16, device="cuda")
        sb = torch.full((ns + 1024,), 7.0, device="cuda")
        y, hf, st = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"], y=big[512:512 + ny].view(B, L, D),
                                  states=sb[512:512 + ns])
        assert (big[:512] == 7).all() and (big[512 + ny:] == 7).all() and (sb[:512] == 7).all() and (sb[512 + ns:] == 7).all()
        g = S.glr_backward(d["x"], d["gate"], d["dy"], st, d["rate"], d["input_gate"], d["dh_final"])
        got = [y.clone(), hf, *(g[k] for k in sorted(g))]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_gradients_against_differences_of_the_operator():
    """The kernels' own forward differenced (fp32, steps of 2^-6 of one whole input's direction)."""
    B, L, D = 1, 60, 16
    d = cuda(make(B, L, D, "f32", True, True, True))
    r = torch.Generator(device="cuda").manual_seed(3)

    def loss(q):
        y, hf, _ = S.glr_forward(q["x"], q["gate"], q["rate"], q["input_gate"], q["h0"])
        return float((y.double() * d["dy"].double()).sum() + (hf.double() * d["dh_final"].double()).sum())
    _, _, st = S.glr_forward(d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"], want_states=True)
    g = S.glr_backward(d["x"], d["gate"], d["dy"], st, d["rate"], d["input_gate"], d["dh_final"])
    for name, grad in (("x", "dx"), ("gate", "dgate"), ("input_gate", "dinput_gate"), ("rate", "drate"), ("h0", "dh0")):
        v = torch.randn(d[name].shape, generator=r, device="cuda")
        if name == "rate":
            v = v * d["rate"]
        f = lambda e: loss(dict(d, **{name: d[name] + e * v}))
        e = 2.0 ** -6
        # fourth-order central difference: truncation e^4 f'''''/30 ~ 2e-9 |f'''''|, rounding: each loss
        # sums ~1000 terms known to ~1e-6, so about 1e-6 sqrt(1000) / e = 2e-3 absolute
        got = (8 * (f(e) - f(-e)) - (f(2 * e) - f(-2 * e))) / (12 * e)
        want = float((g[grad].double() * v.double()).sum())
        assert abs(got - want) <= 1e-2 + 1e-3 * abs(want), (name, got, want)


def test_other_streams_and_graphs():
    d = cuda(make(2, 700, 136, "bf16", True, True, True))
    args = (d["x"], d["gate"], d["rate"], d["input_gate"], d["h0"])

    def both(stream=None):
        y, hf, st = S.glr_forward(*args, want_states=True, stream=stream)
        g = S.glr_backward(d["x"], d["gate"], d["dy"], st, d["rate"], d["input_gate"], d["dh_final"], stream=stream)
        return [y, hf] + [g[k] for k in sorted(g)]
    want = both()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = [], []
    for _ in range(5):   # two streams at once, tensors allocated for each
        a, b = both(s1), both(s2)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, a)) and all(torch.equal(p, q) for p, q in zip(want, b))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    d["x"].mul_(0.5)
    d["dy"].mul_(-2.0)
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    want = both()
    for _, out in graphs:
        assert all(torch.equal(p, q) for p, q in zip(want, out))


def test_the_binding_refuses():
    d = cuda(make(2, 20, 24, "f32", True, True, True))
    x, g = d["x"], d["gate"]
    st = S.new_glr_states(2, 20, 24)
    bad = [dict(gate=g[:, :-1]), dict(gate=g.bfloat16()), dict(gate=g.cpu()), dict(gate=g.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(rate=d["rate"][:-1]), dict(rate=d["rate"].double()), dict(input_gate=g[:1]), dict(h0=d["h0"].bfloat16()),
           dict(h0=d["h0"][:, :-1]), dict(y=x[:1]), dict(h_final=d["h0"].half()), dict(states=st[:-1])]
    for kw in bad:
        with pytest.raises(ValueError):
            S.glr_forward(**dict(dict(x=x, gate=g), **kw))
    with pytest.raises(TypeError):
        S.glr_forward(x.half(), g.half())
    with pytest.raises(ValueError):
        S.glr_forward(x[0], g[0])
    with pytest.raises(S.SscanError) as e:   # y over x
        S.glr_forward(x, g, y=x)
    assert e.value.code == S.ERR_INVALID
    flat = torch.zeros(2 * 20 * 24 + 1, device="cuda")
    with pytest.raises(S.SscanError) as e:
        S.glr_forward(flat[1:].view(2, 20, 24), g)
    assert e.value.code == S.ERR_ALIGN
    for kw in (dict(dy=x[:1]), dict(states=st[:-1]), dict(states=st.view(2, -1)), dict(dh_final=d["h0"].double()),
               dict(rate=d["rate"], workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            S.glr_backward(**dict(dict(x=x, gate=g, dy=x, states=st), **kw))
    with pytest.raises(S.SscanError):
        S.glr_forward(torch.empty(0, 4, 8, device="cuda"), torch.empty(0, 4, 8, device="cuda"))
