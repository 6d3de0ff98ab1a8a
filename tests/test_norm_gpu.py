"""GPU tests of the layer norm against the fp64 oracle, elementwise, with bounds from its arithmetic.

U = 2^-24.  A sum of D terms held by at least 32 threads and joined by a tree is off by at most
g = (D / 32 + 16) U times the sum of the absolute values; every other operation by U, a square root
and a division by U each.  With A = mean |s|, the mean is off by dmu = (g + 2 U) A, the centred value
by dc = dmu + U |s - mu|, the variance V by 2 dmu mean|s - mu| + dmu^2 + (g + 6 U) V, and rstd by
r = dV / (2 (V + eps)) + 3 U relative.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from selective_state_space_32_b200 import sscan as S

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_32_b200 import build
    build.build()
    S.lib()


def make(rows, D, dtype, residual, weight=True, bias=True, seed=0, mean=0.0):
    r = np.random.default_rng(seed + rows * 31 + D)
    f = lambda v: torch.from_numpy(np.asarray(v, np.float32))
    rt = {None: None, "same": DT[dtype], "f32": torch.float32}[residual]
    d = {"x": f(r.standard_normal((rows, D)) + mean).to(DT[dtype]),
         "residual": None if rt is None else f(2 * r.standard_normal((rows, D))).to(rt),
         "weight": f(1 + 0.3 * r.standard_normal(D)) if weight else None,
         "bias": f(r.standard_normal(D)) if bias else None,
         "dy": f(r.standard_normal((rows, D))).to(DT[dtype])}
    d["dresidual"] = None if rt is None else f(r.standard_normal((rows, D))).to(rt)
    return d


def h(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, ref, bound, what):
    got = h(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not got.size:
        return
    over = np.where(got == ref, 0.0, np.abs(got - ref) / np.maximum(bound, 1e-300))
    over = np.where(np.isnan(over), np.inf, over)
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 1.0, f"{what}{i}: got {got[i]!r}, want {ref[i]!r}, bound {bound[i]!r}"


def rounded(ref, err, dt):
    return err + (2.0 ** -8 if dt == torch.bfloat16 else U) * (np.abs(ref) + err)


def stats_bounds(s, rms, eps):
    D = s.shape[1]
    g = (D / 32 + 16) * U
    mu = np.zeros((len(s), 1)) if rms else s.mean(1, keepdims=True)
    c = np.abs(s - mu)
    dmu = 0.0 * mu if rms else (g + 2 * U) * np.abs(s).mean(1, keepdims=True)
    V = (c ** 2).mean(1, keepdims=True)
    dV = 2 * dmu * c.mean(1, keepdims=True) + dmu ** 2 + (g + 6 * U) * V
    r = dV / (2 * (V + eps)) + 3 * U
    return mu, c, dmu, dmu + U * c, r, g


def check(rows, D, dtype, residual, rms, weight=True, bias=True, mean=0.0, eps=EPS, seed=0):
    d = make(rows, D, dtype, residual, weight, bias, seed, mean)
    c = {k: None if v is None else v.cuda() for k, v in d.items()}
    y, s, mu, rstd = S.norm_forward(c["x"], c["weight"], c["bias"], residual=c["residual"], eps=eps, rms=rms)
    if residual is None:
        assert s is c["x"]
    else:
        want_s = (d["x"].float() + d["residual"].float()).to(d["residual"].dtype)
        assert torch.equal(s.cpu(), want_s)
    sv = h(s)
    yr, mr, rr = BO.norm_forward(sv, h(d["weight"]), h(d["bias"]), eps, rms)
    mu0, cen, dmu, dc, r, g = stats_bounds(sv, rms, eps)
    w = np.abs(h(d["weight"])) if weight else 1.0
    z = cen * rr[:, None]
    dz = dc * rr[:, None] * (1 + r) + z * (r + 2 * U)
    err = dz * w + 2 * U * z * w + (U * np.abs(h(d["bias"])) if bias else 0.0)
    close(y, yr, rounded(yr, err, DT[dtype]), "y")
    assert (mu is None) == rms
    if not rms:
        close(mu, mr, np.broadcast_to(dmu, (rows, 1))[:, 0] + U * np.abs(mr), "mean")
    close(rstd, rr, rr * (r[:, 0] + U), "rstd")
    y2 = S.norm_forward(c["x"], c["weight"], c["bias"], residual=c["residual"], eps=eps, rms=rms, want_stats=False)
    assert torch.equal(y, y2[0]) and y2[2] is None and y2[3] is None
    # backward, from the kernel's own statistics: their error is in the bound
    b = S.norm_backward(c["dy"], s, mu, rstd, c["weight"], c["dresidual"], rms=rms, want_dbias=bias)
    dyv, wv = h(d["dy"]), h(d["weight"])
    ds, dw, db = BO.norm_backward(dyv, sv, wv, h(d["dresidual"]), eps, rms)
    W = np.abs(dyv * (1.0 if wv is None else wv))
    m2 = np.abs(((dyv * (1.0 if wv is None else wv)) * (sv - mu0) * rr[:, None]).mean(1, keepdims=True))
    a1, a2 = W.mean(1, keepdims=True), (W * z).mean(1, keepdims=True)
    d2 = (W * dz).mean(1, keepdims=True) + (g + 4 * U) * a2
    inner = U * W + (0.0 if rms else (g + 2 * U) * a1) + dz * m2 + z * d2 + dz * d2 + 3 * U * (W + a1 + z * m2)
    full = W + (0.0 if rms else a1) + z * m2
    err = rr[:, None] * (inner * (1 + r) + full * (r + 2 * U))
    if residual is not None:
        err = err + U * np.abs(h(d["dresidual"]))
    close(b["dx"], ds, rounded(ds, err, DT[dtype]), "dx")
    close(b["dresidual"], ds, rounded(ds, err, s.dtype), "dresidual")
    assert (b["dx"] is b["dresidual"]) == (s.dtype == DT[dtype])
    # sums over rows: at most `rows` additions of any term
    if weight:
        close(b["dweight"], dw, (np.abs(dyv) * dz).sum(0) + (rows + 16) * U * (np.abs(dyv) * z).sum(0), "dweight")
    else:
        assert b["dweight"] is None
    if bias:
        close(b["dbias"], db, (rows + 16) * U * np.abs(dyv).sum(0), "dbias")
    else:
        assert b["dbias"] is None


WIDTHS = [1, 2, 3, 7, 8, 31, 64, 65, 100, 128, 250, 256, 257, 512, 768, 777, 1000, 1024, 1032, 2048, 2050, 2560, 4096, 4104, 5120,
          5121, 8192, 8200, 12288, 20000]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, rms):
    for k, (dtype, residual) in enumerate((("f32", None), ("f32", "same"), ("bf16", None), ("bf16", "same"), ("bf16", "f32"))):
        check(5, D, dtype, residual, rms, weight=(D + k) % 3 != 0, bias=(D + k) % 2 == 0)


@pytest.mark.parametrize("rows", [1, 2, 3, 17, 147, 148, 149, 295, 296, 297, 1000, 3001])
def test_rows(rows):
    check(rows, 72, "bf16", "same", False)
    check(rows, 65, "f32", None, False)
    check(rows, 640, "bf16", "f32", True, bias=False)


@pytest.mark.parametrize("rows,D,dtype,residual", [(149, 12288, "bf16", "same"), (700, 10248, "bf16", "f32"), (743, 6001, "bf16", None),
                                                   (297, 16384, "f32", "same"), (1300, 5121, "f32", None), (2, 40001, "bf16", "same")])
def test_rows_in_several_passes(rows, D, dtype, residual):
    """Rows too long for a block's registers: one row a block, several, and a last batch of fewer."""
    check(rows, D, dtype, residual, False)


@pytest.mark.parametrize("D", [257, 258, 301, 777, 2050, 4100, 5121])
@pytest.mark.parametrize("dtype,residual", [("bf16", None), ("bf16", "f32"), ("bf16", "same"), ("f32", "same")])
def test_rows_off_the_boundary(D, dtype, residual):
    """Rows that begin inside a vector, for blocks of one row and of several; the rows next to a
    bad one, which share its first and last vectors, are the same without it."""
    check(1203 if D < 1000 else 800, D, dtype, residual, D % 3 == 0, bias=D % 2 == 0)
    d = {k: None if v is None else v.cuda() for k, v in make(700, D, dtype, residual).items()}
    run = lambda x, r, dy: (lambda f: (f, S.norm_backward(dy, f[1], f[2], f[3], d["weight"], d["dresidual"], want_dbias=True)))(
        S.norm_forward(x, d["weight"], d["bias"], residual=r))
    f, b = run(d["x"], d["residual"], d["dy"])
    bad = [0, 5, 342, 343, 699]
    x, dy = d["x"].clone(), d["dy"].clone()
    x[bad] = float("nan")
    dy[bad] = float("inf")
    f2, b2 = run(x, d["residual"], dy)
    keep = [i for i in range(700) if i not in bad]
    for p, q in zip(f + (b["dx"], b["dresidual"]), f2 + (b2["dx"], b2["dresidual"])):
        assert torch.equal(p[keep], q[keep])


@pytest.mark.parametrize("mean", [0.0, 30.0, 1000.0])
def test_a_mean_far_from_zero(mean):
    check(6, 640, "f32", None, False, mean=mean)
    check(6, 4096, "f32", "same", False, mean=mean)


def test_constant_rows_and_rows_of_zeros():
    for D in (64, 100, 4096):
        x = torch.full((3, D), 2.0, device="cuda")
        x[1] = 0.0
        y, _, mu, rstd = S.norm_forward(x)
        assert not y.any() and torch.equal(mu.cpu(), torch.tensor([2.0, 0.0, 2.0]))
        assert torch.allclose(rstd, torch.full((3,), EPS ** -0.5, device="cuda"), rtol=1e-6)
        y = S.norm_forward(x[1:2], rms=True)[0]
        assert not y.any()


def test_a_bad_row_stays_a_bad_row():
    for D in (72, 2048, 5121):
        d = make(40, D, "f32", "same")
        c = {k: v.cuda() for k, v in d.items()}
        y, s, mu, rstd = S.norm_forward(c["x"], c["weight"], c["bias"], residual=c["residual"])
        b = S.norm_backward(c["dy"], s, mu, rstd, c["weight"], c["dresidual"])
        x = c["x"].clone()
        x[7, D // 2] = float("nan")
        x[8, 0] = float("inf")
        y2, s2, mu2, rstd2 = S.norm_forward(x, c["weight"], c["bias"], residual=c["residual"])
        b2 = S.norm_backward(c["dy"], s2, mu2, rstd2, c["weight"], c["dresidual"])
        keep = [i for i in range(40) if i not in (7, 8)]
        assert torch.equal(y[keep], y2[keep]) and torch.equal(b["dx"][keep], b2["dx"][keep])
        assert torch.isnan(y2[7]).all() and not torch.isfinite(y2[8, 0])


def test_leading_dimensions_and_no_rows():
    x = torch.randn(2, 3, 5, 48, device="cuda")
    y, s, mu, rstd = S.norm_forward(x)
    assert y.shape == x.shape and mu.shape == (2, 3, 5) and rstd.shape == (2, 3, 5)
    flat = S.norm_forward(x.view(30, 48))
    assert torch.equal(flat[0].view_as(y), y)
    b = S.norm_backward(x, s, mu, rstd, want_dbias=True)
    assert torch.equal(b["dx"].view(30, 48), S.norm_backward(x.view(30, 48), x.view(30, 48), mu.view(30), rstd.view(30))["dx"])
    one = S.norm_forward(x[0, 0, 0])
    assert one[0].shape == (48,) and one[2].shape == () and torch.equal(one[0], y[0, 0, 0])
    e = torch.empty(0, 48, device="cuda")
    w = torch.ones(48, device="cuda")
    y, s, mu, rstd = S.norm_forward(e, w)
    b = S.norm_backward(e, e, mu, rstd, w, want_dbias=True)
    assert y.shape == (0, 48) and not b["dweight"].any() and not b["dbias"].any()


def test_the_same_call_gives_the_same_bits_on_streams_and_in_graphs():
    d = make(2003, 2048, "bf16", "f32")
    c = {k: v.cuda() for k, v in d.items()}

    def both(stream=None):
        y, s, mu, rstd = S.norm_forward(c["x"], c["weight"], c["bias"], residual=c["residual"], stream=stream)
        b = S.norm_backward(c["dy"], s, mu, rstd, c["weight"], c["dresidual"], want_dbias=True, stream=stream)
        return [y, s, mu, rstd] + [b[k] for k in sorted(b)]
    want = both()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a, b = both(s1), both(s2)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, a)) and all(torch.equal(p, q) for p, q in zip(want, b))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    c["x"].mul_(0.5)
    c["dy"].mul_(-2.0)
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    want = both()
    for _, out in graphs:
        assert all(torch.equal(p, q) for p, q in zip(want, out))


def test_gradients_against_differences_of_the_operator():
    c = {k: v.cuda() for k, v in make(4, 40, "f32", "same").items()}
    gen = torch.Generator(device="cuda").manual_seed(3)

    def loss(q):
        y, s, _, _ = S.norm_forward(q["x"], q["weight"], q["bias"], residual=q["residual"])
        return float((y.double() * c["dy"].double()).sum() + (s.double() * c["dresidual"].double()).sum())
    y, s, mu, rstd = S.norm_forward(c["x"], c["weight"], c["bias"], residual=c["residual"])
    b = S.norm_backward(c["dy"], s, mu, rstd, c["weight"], c["dresidual"], want_dbias=True)
    for name, grad in (("x", "dx"), ("residual", "dresidual"), ("weight", "dweight"), ("bias", "dbias")):
        v = torch.randn(c[name].shape, generator=gen, device="cuda")
        f = lambda e: loss(dict(c, **{name: c[name] + e * v}))
        e = 2.0 ** -6
        # fourth-order central difference; each loss sums 320 terms known to ~4e-7: 4e-7 sqrt(320) 1.5 / e = 7e-4
        got = (8 * (f(e) - f(-e)) - (f(2 * e) - f(-2 * e))) / (12 * e)
        want = float((b[grad].double() * v.double()).sum())
        assert abs(got - want) <= 4e-3 + 1e-4 * abs(want), (name, got, want)


@pytest.mark.parametrize("rows,D", [(5, 24), (33, 65), (7, 640), (3, 777), (9, 2048), (300, 100)])
def test_nothing_outside_the_outputs_is_written(rows, D):
    """Every output through the C ABI inside a larger buffer: the rest keeps its values."""
    import ctypes
    lib, n = S.lib(), rows * D
    d = {k: v.cuda() for k, v in make(rows, D, "bf16", "f32").items()}
    p = lambda t, off=0: ctypes.c_void_p(t.data_ptr() + off)
    pad = 64
    held = []

    def inside(count, dt):
        t = torch.full((count + 2 * pad,), 5.0, dtype=dt, device="cuda")
        held.append((t, count))
        return p(t, pad * t.element_size()), t[pad:pad + count]
    y, _ = inside(n, torch.bfloat16)
    s, sv = inside(n, torch.float32)
    mean, mv = inside(rows, torch.float32)
    rstd, rv = inside(rows, torch.float32)
    assert lib.sscan_norm_forward(rows, D, S.BF16, S.NORM_RESIDUAL_F32, EPS, p(d["x"]), p(d["residual"]), p(d["weight"]),
                                  p(d["bias"]), y, s, mean, rstd, None) == S.OK
    ds, _ = inside(n, torch.float32)
    dx, _ = inside(n, torch.bfloat16)
    dw, _ = inside(D, torch.float32)
    db, _ = inside(D, torch.float32)
    ws = int(lib.sscan_norm_backward_workspace_bytes(rows, D))
    w, _ = inside(ws // 4, torch.float32)
    torch.cuda.synchronize()
    assert lib.sscan_norm_backward(rows, D, S.BF16, S.NORM_RESIDUAL_F32, p(d["dy"]), s, mean, rstd, p(d["weight"]),
                                   p(d["dresidual"]), ds, dx, dw, db, w, None) == S.OK
    torch.cuda.synchronize()
    for t, count in held:
        assert (t[:pad] == 5).all() and (t[pad + count:] == 5).all()
    want = S.norm_forward(d["x"], d["weight"], d["bias"], residual=d["residual"])
    assert torch.equal(want[1].view(-1), sv) and torch.equal(want[2], mv) and torch.equal(want[3], rv)


def test_the_binding_refuses():
    x = torch.randn(4, 24, device="cuda")
    w = torch.ones(24, device="cuda")
    for kw in (dict(weight=w[:-1]), dict(weight=w.bfloat16()), dict(bias=w.cpu()), dict(residual=x[:2]), dict(residual=x.t().contiguous().t())):
        with pytest.raises(ValueError):
            S.norm_forward(x, **kw)
    with pytest.raises(TypeError):
        S.norm_forward(x, residual=x.bfloat16())
    with pytest.raises(TypeError):
        S.norm_forward(x.half())
    with pytest.raises(S.SscanError):
        S.norm_forward(x, eps=-1.0)
    with pytest.raises(S.SscanError):
        S.norm_forward(torch.empty(4, 0, device="cuda"))
    y, s, mu, rstd = S.norm_forward(x)
    for a, kw in (((x, s, None, rstd), {}), ((x, s, mu, rstd), dict(rms=True)), ((x, s[:2], mu, rstd), {}),
                  ((x, s, mu[:2], rstd), {}), ((x, s, mu, rstd), dict(dresidual=x.bfloat16())),
                  ((x, s, mu, rstd), dict(want_dbias=True, workspace=torch.empty(3, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(ValueError):
            S.norm_backward(*a, **kw)
