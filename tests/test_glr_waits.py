"""The report of a wait that gives up: the blocks of a cluster wait for each other's maps, and a
wait without tries gives up at once (nothing hangs: every block still ends its walk)."""
import ctypes

import pytest
import torch

from selective_state_space_32_b200 import build as B
from selective_state_space_32_b200 import sscan as S

P = [ctypes.c_void_p(1 << 20 | k << 16) for k in range(1, 20)]  # distinct aligned addresses, never dereferenced


def _off(p, n):
    return ctypes.c_void_p(p.value + n)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.lib()


def test_the_status_word_is_checked(lib):
    def fwd(status, h0=None, hf=None):
        return lib.sscan_glr_forward_checked(1, 4, 8, S.F32, P[0], P[1], None, None, h0, P[2], hf, P[3], status, 5, None)

    def bwd(status):
        return lib.sscan_glr_backward_checked(1, 4, 8, S.F32, P[0], P[1], None, P[6], P[2], P[3], None, P[4], P[5], None,
                                              P[7], None, P[8], status, 5, None)
    assert fwd(_off(P[9], 2)) == S.ERR_ALIGN and bwd(_off(P[9], 1)) == S.ERR_ALIGN
    for k in range(4):
        assert fwd(_off(P[k], 28)) == S.ERR_INVALID     # inside x, gate, y, the states
    assert fwd(P[10], h0=P[10]) == S.ERR_INVALID and fwd(P[10], hf=P[10]) == S.ERR_INVALID
    assert fwd(P[10], h0=P[10], hf=P[10]) == S.ERR_INVALID
    for k in range(8):
        assert bwd(_off(P[k], 28)) == S.ERR_INVALID     # inside an input or an output
    assert bwd(_off(P[8], 8)) == S.ERR_WORKSPACE
    assert lib.sscan_glr_forward_checked(0, 4, 8, S.F32, P[0], P[1], None, None, None, P[2], None, None, P[9], 0,
                                         None) == S.ERR_INVALID


@pytest.fixture
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    return S.lib()


def _inputs(Bn, L, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(L)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x, gate, ig, dy = (n(Bn, L, D).to(dtype) for _ in range(4))
    return x, gate, ig, dy, 0.01 + 0.5 * torch.rand(D, device="cuda", generator=g), n(Bn, D)


def _checked(lib, t, status, tries, h0=None, h_final=None):
    x, gate, ig, dy, rate, _ = t
    Bn, L, D = x.shape
    code = S.BF16 if x.dtype == torch.bfloat16 else S.F32
    a = lambda v: None if v is None else v.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    y, states = torch.zeros_like(x), S.new_glr_states(Bn, L, D).zero_()
    rc = lib.sscan_glr_forward_checked(Bn, L, D, code, a(x), a(gate), a(ig), a(rate), a(h0), a(y), a(h_final), a(states),
                                       a(status[:1]), tries, st)
    assert rc == S.OK
    ws = torch.empty(int(lib.sscan_glr_backward_workspace_bytes(Bn, L, D)), dtype=torch.uint8, device="cuda")
    d = [torch.zeros_like(x) for _ in range(3)] + [torch.zeros_like(rate)]
    rc = lib.sscan_glr_backward_checked(Bn, L, D, code, a(x), a(gate), a(ig), a(rate), a(states), a(dy), None, *map(a, d),
                                        None, a(ws), a(status[1:]), tries, st)
    assert rc == S.OK
    torch.cuda.synchronize()
    return [y] + d


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,L,D,dtype", [
    (1, 20000, 64, torch.bfloat16),    # clusters of 16 blocks of 8 warps
    (1, 9000, 96, torch.float32),
    (2, 3000, 1024, torch.bfloat16),   # clusters of 8
    (8, 600, 1536, torch.bfloat16),    # of 2
    (1, 2000, 101, torch.bfloat16),    # rows that are loaded directly
])
def test_a_wait_that_gives_up_is_reported(cuda_lib, Bn, L, D, dtype):
    t = _inputs(Bn, L, D, dtype)
    x, gate, ig, dy, rate, h0 = t
    want, _, states = S.glr_forward(x, gate, rate, ig, want_states=True)
    status = torch.tensor([8, 8], dtype=torch.int32, device="cuda")   # bits that are there stay
    for tries in (S._ALL_TRIES, 0, S._ALL_TRIES):
        out = _checked(cuda_lib, t, status, tries)
        if tries:
            assert status.tolist() == [8, 8] and torch.equal(out[0], want) and all(torch.isfinite(q).all() for q in out)
        else:
            assert status.tolist() == [9, 9]
            assert all(torch.isnan(q).all() for q in out)
            status.fill_(8)
    h = h0.clone()
    _checked(cuda_lib, t, status, 0, h, h)   # the state in place is lost with the outputs
    assert torch.isnan(h).all() and status.tolist() == [9, 9]
    again = S.glr_forward(x, gate, rate, ig)[0]
    assert torch.equal(again, want)


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,L,D,dtype", [(3, 300, 4096, torch.float32), (4, 5, 200, torch.bfloat16), (70, 17, 8000, torch.float32)])
def test_a_walk_of_one_block_waits_for_nobody(cuda_lib, Bn, L, D, dtype):
    t = _inputs(Bn, L, D, dtype)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = _checked(cuda_lib, t, status, 0)
    assert not status.any()
    for a, b in zip(out, _checked(cuda_lib, t, status, S._ALL_TRIES)):
        assert torch.equal(a, b) and torch.isfinite(a).all()


@pytest.mark.gpu
def test_the_binding_takes_a_status(cuda_lib):
    x, gate, ig, dy, rate, h0 = _inputs(2, 3000, 96, torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = S.glr_forward(x, gate, rate, ig, h0, want_states=True)
    b = S.glr_forward(x, gate, rate, ig, h0, want_states=True, status=status)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = (S.glr_backward(x, gate, dy, a[2], rate, ig, status=s, stream=torch.cuda.current_stream()) for s in (None, status))
    assert all(torch.equal(a[k], b[k]) for k in a) and not status.any()
    for bad in (status.float(), status.cpu(), torch.zeros(2, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            S.glr_forward(x, gate, rate, ig, h0, status=bad)
        with pytest.raises(ValueError):
            S.glr_backward(x, gate, dy, S.new_glr_states(2, 3000, 96), rate, ig, status=bad)
