"""GPU tests of the norm's backward pass where its blocks walk several rows through a ring of one row,
and on both sides of the widths at which the ring changes.  Bounds as in test_norm_gpu.py."""
import pytest
import torch

from selective_state_space_32_b200 import sscan as S
from tests.test_norm_gpu import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_32_b200 import build
    build.build()
    S.lib()


# 700 rows on 148 blocks at most.  The ring holds two rows up to about 8045 values (fp32) and 9386 (bf16
# with an fp32 residual), one up to 10240; longer rows are read twice.
CASES = ([("f32", "same", D) for D in (8041, 8044, 8047, 8048, 8192, 9001, 9002, 10237, 10239, 10240, 10241, 10244)]
         + [("bf16", "f32", D) for D in (9380, 9384, 9391, 9392, 9600, 9601, 10001, 10233, 10235, 10240, 10248)])


@pytest.mark.parametrize("dtype,residual,D", CASES)
def test_rows_that_fill_shared_memory(dtype, residual, D):
    check(700, D, dtype, residual, D % 2 == 0, bias=D % 3 != 0)


@pytest.mark.parametrize("dtype,residual,D", [("f32", "same", 9001), ("f32", "same", 8192), ("bf16", "f32", 9601), ("bf16", "f32", 9600)])
def test_neighbours_of_bad_rows_and_the_same_bits(dtype, residual, D):
    d = {k: None if v is None else v.cuda() for k, v in make(700, D, dtype, residual).items()}

    def run(x, dy):
        f = S.norm_forward(x, d["weight"], d["bias"], residual=d["residual"])
        b = S.norm_backward(dy, f[1], f[2], f[3], d["weight"], d["dresidual"], want_dbias=True)
        return f, b
    f, b = run(d["x"], d["dy"])
    for _ in range(3):
        f1, b1 = run(d["x"], d["dy"])
        assert all(torch.equal(p, q) for p, q in zip(f, f1)) and all(torch.equal(b[k], b1[k]) for k in b)
    bad = [0, 147, 148, 300, 699]
    x, dy = d["x"].clone(), d["dy"].clone()
    x[bad], dy[bad] = float("nan"), float("inf")
    f2, b2 = run(x, dy)
    keep = [i for i in range(700) if i not in bad]
    for p, q in zip(f + (b["dx"], b["dresidual"]), f2 + (b2["dx"], b2["dresidual"])):
        assert torch.equal(p[keep], q[keep])
        assert not torch.isfinite(q[bad]).any()


@pytest.mark.parametrize("rows,dtype,residual,D", [(700, "f32", "same", 10244), (700, "bf16", "f32", 12288), (3, "bf16", None, 40001),
                                                   (601, "bf16", "same", 10240), (601, "f32", None, 777)])
def test_the_workspace_is_as_large_as_stated(rows, dtype, residual, D):
    """A workspace of just that size inside a larger buffer: the rest keeps its values, the gradients their bits."""
    d = {k: None if v is None else v.cuda() for k, v in make(rows, D, dtype, residual).items()}
    y, s, mu, rstd = S.norm_forward(d["x"], d["weight"], d["bias"], residual=d["residual"])
    want = S.norm_backward(d["dy"], s, mu, rstd, d["weight"], d["dresidual"], want_dbias=True)
    n = int(S.lib().sscan_norm_backward_workspace_bytes(rows, D))
    big = torch.full((n + 8192,), 7, dtype=torch.uint8, device="cuda")
    got = S.norm_backward(d["dy"], s, mu, rstd, d["weight"], d["dresidual"], want_dbias=True, workspace=big[4096:4096 + n])
    assert all(torch.equal(want[k], got[k]) for k in want)
    assert (big[:4096] == 7).all() and (big[4096 + n:] == 7).all()
