"""Argument checks of the recurrent block's operators that come before any CUDA call
(no GPU: every case below is refused, or has nothing to do)."""
import ctypes

import pytest
import torch

from selective_state_space_32_b200 import build as B
from selective_state_space_32_b200 import sscan as S

P = [ctypes.c_void_p(1 << 20 | k << 16) for k in range(1, 20)]  # distinct aligned addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.lib()


def _fwd(lib, B=1, L=4, D=8, dtype=S.F32, x=P[0], gate=P[1], ig=None, rate=None, h0=None, y=P[2], hf=None, states=None):
    return lib.sscan_glr_forward(B, L, D, dtype, x, gate, ig, rate, h0, y, hf, states, None)


def _off(p, n):
    return ctypes.c_void_p(p.value + n)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), S.ERR_INVALID), (dict(D=0), S.ERR_INVALID), (dict(L=-1), S.ERR_INVALID), (dict(dtype=7), S.ERR_INVALID),
    (dict(B=1 << 31), S.ERR_UNSUPPORTED), (dict(D=1 << 31), S.ERR_UNSUPPORTED), (dict(L=1 << 50), S.ERR_UNSUPPORTED),
    (dict(B=1 << 30, D=1 << 10), S.ERR_UNSUPPORTED),
    (dict(x=None), S.ERR_INVALID), (dict(gate=None), S.ERR_INVALID), (dict(y=None), S.ERR_INVALID),
    (dict(x=_off(P[0], 4)), S.ERR_ALIGN), (dict(gate=_off(P[1], 8)), S.ERR_ALIGN), (dict(y=_off(P[2], 2)), S.ERR_ALIGN),
    (dict(ig=_off(P[3], 2)), S.ERR_ALIGN), (dict(rate=_off(P[3], 4)), S.ERR_ALIGN), (dict(h0=_off(P[3], 4)), S.ERR_ALIGN),
    (dict(hf=_off(P[3], 4)), S.ERR_ALIGN), (dict(states=_off(P[3], 4)), S.ERR_ALIGN),
    (dict(y=P[0]), S.ERR_INVALID), (dict(y=_off(P[1], 112)), S.ERR_INVALID),         # y over x, y over gate's last 16 bytes
    (dict(ig=P[3], y=P[3]), S.ERR_INVALID), (dict(states=P[2]), S.ERR_INVALID), (dict(hf=P[2]), S.ERR_INVALID),
    (dict(hf=P[0]), S.ERR_INVALID), (dict(h0=P[4], hf=_off(P[4], 16)), S.ERR_INVALID),  # h_final over part of h0
    (dict(h0=P[2], hf=P[2]), S.ERR_INVALID), (dict(h0=P[0], hf=P[0]), S.ERR_INVALID),   # in place, but over y or x
])
def test_glr_forward_refuses(lib, kw, want):
    assert _fwd(lib, **kw) == want


def test_glr_backward_refuses(lib):
    def bwd(B=1, L=4, D=8, dtype=S.F32, x=P[0], gate=P[1], ig=None, rate=None, states=P[2], dy=P[3], dhf=None, dx=P[4],
            dgate=P[5], dig=None, drate=None, dh0=None, ws=None):
        return lib.sscan_glr_backward(B, L, D, dtype, x, gate, ig, rate, states, dy, dhf, dx, dgate, dig, drate, dh0, ws, None)
    for k in ("x", "gate", "states", "dy", "dx", "dgate"):
        assert bwd(**{k: None}) == S.ERR_INVALID, k
    assert bwd(B=0) == S.ERR_INVALID and bwd(dtype=2) == S.ERR_INVALID and bwd(L=1 << 50) == S.ERR_UNSUPPORTED
    assert bwd(ig=P[6]) == S.ERR_INVALID and bwd(dig=P[6]) == S.ERR_INVALID       # a gate without its gradient, and back
    assert bwd(rate=P[6]) == S.ERR_INVALID and bwd(drate=P[6]) == S.ERR_INVALID
    assert bwd(rate=P[6], drate=P[7]) == S.ERR_WORKSPACE                          # the rate's sums need one
    assert bwd(rate=P[6], drate=P[7], ws=P[0]) == S.ERR_WORKSPACE and bwd(rate=P[6], drate=P[7], ws=P[4]) == S.ERR_WORKSPACE
    assert bwd(rate=P[6], drate=P[7], ws=_off(P[8], 8)) == S.ERR_ALIGN
    assert bwd(dx=P[3]) == S.ERR_INVALID and bwd(dx=P[5]) == S.ERR_INVALID and bwd(dh0=P[2]) == S.ERR_INVALID
    assert bwd(dhf=P[6], dh0=P[6]) == S.ERR_INVALID and bwd(dh0=_off(P[6], 4)) == S.ERR_ALIGN


def test_norm_refuses(lib):
    def fwd(rows=4, D=8, dtype=S.BF16, flags=0, eps=1e-5, x=P[0], r=None, w=None, b=None, y=P[1], ro=None, mean=None, rstd=None):
        return lib.sscan_norm_forward(rows, D, dtype, flags, eps, x, r, w, b, y, ro, mean, rstd, None)
    assert fwd(D=0) == S.ERR_INVALID and fwd(rows=-1) == S.ERR_INVALID and fwd(dtype=5) == S.ERR_INVALID
    assert fwd(flags=4) == S.ERR_INVALID and fwd(rows=1 << 45) == S.ERR_UNSUPPORTED
    assert fwd(eps=-1.0) == S.ERR_INVALID and fwd(eps=float("nan")) == S.ERR_INVALID and fwd(eps=float("inf")) == S.ERR_INVALID
    assert fwd(x=None) == S.ERR_INVALID and fwd(y=None) == S.ERR_INVALID
    assert fwd(r=P[2]) == S.ERR_INVALID and fwd(ro=P[2]) == S.ERR_INVALID          # residual and its sum go together
    assert fwd(flags=S.NORM_RMS, mean=P[2]) == S.ERR_INVALID
    assert fwd(y=P[0]) == S.ERR_INVALID and fwd(r=P[2], ro=P[2]) == S.ERR_INVALID and fwd(r=P[2], ro=P[1]) == S.ERR_INVALID
    assert fwd(w=_off(P[2], 4)) == S.ERR_ALIGN and fwd(rstd=_off(P[2], 8)) == S.ERR_ALIGN
    assert fwd(rows=0, x=None, y=None) == S.OK

    def bwd(rows=4, D=8, dtype=S.BF16, flags=0, dy=P[0], s=P[1], mean=P[2], rstd=P[3], w=P[4], dr=None, ds=P[5], dx=None,
            dw=None, db=None, ws=None):
        return lib.sscan_norm_backward(rows, D, dtype, flags, dy, s, mean, rstd, w, dr, ds, dx, dw, db, ws, None)
    for k in ("dy", "s", "mean", "rstd", "ds"):
        assert bwd(**{k: None}) == S.ERR_INVALID, k
    assert bwd(flags=S.NORM_RMS) == S.ERR_INVALID                                   # a mean with rms
    assert bwd(dx=P[6]) == S.ERR_INVALID                                            # ds has that type already
    assert bwd(dtype=S.F32, flags=S.NORM_RESIDUAL_F32, dx=P[6]) == S.ERR_INVALID
    assert bwd(w=None, dw=P[6]) == S.ERR_INVALID
    assert bwd(dw=P[6]) == S.ERR_WORKSPACE and bwd(db=P[6]) == S.ERR_WORKSPACE and bwd(db=P[6], ws=P[5]) == S.ERR_WORKSPACE
    assert bwd(ds=P[0]) == S.ERR_INVALID and bwd(dr=P[5]) == S.ERR_INVALID and bwd(ds=_off(P[5], 2)) == S.ERR_ALIGN


def test_sizes_of_buffers(lib):
    assert lib.sscan_glr_states_bytes(0, 4, 8) == 0 and lib.sscan_glr_states_bytes(2, 0, 8) == 0
    assert lib.sscan_glr_states_bytes(2, 100, 8) > 0 and lib.sscan_glr_states_bytes(2, 100, 8) % 4 == 0
    assert lib.sscan_glr_backward_workspace_bytes(0, 4, 8) == 0 and lib.sscan_glr_backward_workspace_bytes(1, 0, 8) == 0
    assert lib.sscan_glr_backward_workspace_bytes(2, 100, 8) >= 32
    # a row of D sums per block: one block a batch row where there are many, at most 16
    assert lib.sscan_glr_backward_workspace_bytes(65536, 4, 64) == 65536 * 64 * 4
    assert lib.sscan_glr_backward_workspace_bytes(1, 1 << 20, 64) == 16 * 64 * 4
    assert lib.sscan_norm_backward_workspace_bytes(0, 8) == 0 and lib.sscan_norm_backward_workspace_bytes(5, 8) >= 64


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        S.glr_forward(x, x)
    with pytest.raises(ValueError):
        S.glr_backward(x, x, x, torch.zeros(8))
    with pytest.raises(ValueError):
        S.norm_forward(x)
    with pytest.raises(ValueError):
        S.norm_backward(x, x, torch.zeros(1, 4), torch.zeros(1, 4))
