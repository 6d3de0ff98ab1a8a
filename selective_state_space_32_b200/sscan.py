"""Thin ctypes binding of the C ABI in ``include/sscan.h`` (libsscan.so).

Argument marshalling only: every step of the selective-scan forward runs in the
CUDA library.  PyTorch supplies device memory and the current stream.  There is
no fallback: if the library is missing or the call fails, this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsscan.so")

F32, BF16 = 0, 1
ZOH = 1
DELTA_SOFTPLUS = 2
NORM_RMS, NORM_RESIDUAL_F32 = 1, 2
OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_ALIGN, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(7)

SYMBOLS = ("sscan_plan_create", "sscan_plan_destroy", "sscan_workspace_bytes", "sscan_forward",
           "sscan_get_status", "sscan_status_string", "sscan_plan_describe", "sscan_version",
           "sscan_forward_noalloc", "sscan_noalloc_status", "sscan_forward_gated", "sscan_backward",
           "sscan_backward_workspace_bytes", "sscan_ssd_forward", "sscan_backward_gated",
           "sscan_host_workspace_bytes", "sscan_forward_host", "sscan_glr_states_bytes", "sscan_glr_forward",
           "sscan_glr_forward_checked", "sscan_glr_backward_workspace_bytes", "sscan_glr_backward",
           "sscan_glr_backward_checked", "sscan_norm_forward",
           "sscan_norm_backward_workspace_bytes", "sscan_norm_backward")


class SscanError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} (code {code})")
        self.code = code


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Open libsscan.so (built in-tree by ``python -m selective_state_space_32_b200.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                                   "`python -m selective_state_space_32_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, ip, u32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_uint32, ctypes.c_size_t)
            L.sscan_plan_create.argtypes = [ctypes.POINTER(vp), i64, i64, i64, i64, ip, u32]
            L.sscan_plan_create.restype = ip
            L.sscan_plan_destroy.argtypes = [vp]
            L.sscan_plan_destroy.restype = None
            L.sscan_workspace_bytes.argtypes = [vp]
            L.sscan_workspace_bytes.restype = sz
            L.sscan_forward.argtypes = [vp] * 11
            L.sscan_forward.restype = ip
            L.sscan_get_status.argtypes = [vp, vp]
            L.sscan_get_status.restype = ip
            L.sscan_status_string.argtypes = [ip]
            L.sscan_status_string.restype = ctypes.c_char_p
            L.sscan_plan_describe.argtypes = [vp, ctypes.c_char_p, sz]
            L.sscan_plan_describe.restype = ip
            L.sscan_version.argtypes = []
            L.sscan_version.restype = ip
            L.sscan_forward_noalloc.argtypes = [i64, i64, i64, i64, ip, u32] + [vp] * 9
            L.sscan_forward_noalloc.restype = ip
            L.sscan_noalloc_status.argtypes = [vp]
            L.sscan_noalloc_status.restype = ip
            L.sscan_forward_gated.argtypes = [vp] * 13
            L.sscan_forward_gated.restype = ip
            L.sscan_backward.argtypes = [i64, i64, i64, i64, ip, u32] + [vp] * 16
            L.sscan_backward.restype = ip
            L.sscan_backward_workspace_bytes.argtypes = [i64, i64, i64, i64]
            L.sscan_backward_workspace_bytes.restype = sz
            L.sscan_ssd_forward.argtypes = [i64, i64, i64, i64, i64] + [vp] * 10
            L.sscan_ssd_forward.restype = ip
            L.sscan_backward_gated.argtypes = [i64, i64, i64, i64, ip, u32] + [vp] * 20
            L.sscan_backward_gated.restype = ip
            L.sscan_host_workspace_bytes.argtypes = [vp]
            L.sscan_host_workspace_bytes.restype = sz
            L.sscan_forward_host.argtypes = [vp] * 13
            L.sscan_forward_host.restype = ip
            L.sscan_glr_states_bytes.argtypes = [i64, i64, i64]
            L.sscan_glr_states_bytes.restype = sz
            L.sscan_glr_forward.argtypes = [i64, i64, i64, ip] + [vp] * 9
            L.sscan_glr_forward.restype = ip
            L.sscan_glr_forward_checked.argtypes = [i64, i64, i64, ip] + [vp] * 9 + [u32, vp]
            L.sscan_glr_forward_checked.restype = ip
            L.sscan_glr_backward_workspace_bytes.argtypes = [i64, i64, i64]
            L.sscan_glr_backward_workspace_bytes.restype = sz
            L.sscan_glr_backward.argtypes = [i64, i64, i64, ip] + [vp] * 14
            L.sscan_glr_backward.restype = ip
            L.sscan_glr_backward_checked.argtypes = [i64, i64, i64, ip] + [vp] * 14 + [u32, vp]
            L.sscan_glr_backward_checked.restype = ip
            L.sscan_norm_forward.argtypes = [i64, i64, ip, u32, ctypes.c_float] + [vp] * 9
            L.sscan_norm_forward.restype = ip
            L.sscan_norm_backward_workspace_bytes.argtypes = [i64, i64]
            L.sscan_norm_backward_workspace_bytes.restype = sz
            L.sscan_norm_backward.argtypes = [i64, i64, ip, u32] + [vp] * 12
            L.sscan_norm_backward.restype = ip
            _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().sscan_status_string(int(code)).decode()


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {dt} (float32 or bfloat16)")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class Plan:
    """A sscan_plan for one (B, L, D, N, dtype, zoh, delta_softplus) shape on the current device."""

    def __init__(self, B: int, L: int, D: int, N: int, dtype: torch.dtype = torch.float32,
                 zoh: bool = False, delta_softplus: bool = False):
        self.shape = (int(B), int(L), int(D), int(N))
        self.dtype = dtype
        self.zoh = bool(zoh)
        self.delta_softplus = bool(delta_softplus)
        h = ctypes.c_void_p()
        rc = lib().sscan_plan_create(ctypes.byref(h), *self.shape, _dtype_code(dtype),
                                     (ZOH if zoh else 0) | (DELTA_SOFTPLUS if delta_softplus else 0))
        if rc != OK:
            raise SscanError(rc, "sscan_plan_create")
        self._h = h
        self.workspace_bytes = int(lib().sscan_workspace_bytes(h))

    def close(self):
        if getattr(self, "_h", None):
            lib().sscan_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def describe(self) -> str:
        buf = ctypes.create_string_buffer(512)
        lib().sscan_plan_describe(self._h, buf, 512)
        return buf.value.decode()

    def new_workspace(self, device=None) -> Optional[torch.Tensor]:
        if self.workspace_bytes == 0:
            return None
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device or "cuda")

    def forward(self, u, delta, A, B, C, h0=None, y=None, h_final=None, workspace=None,
                want_final: bool = True, stream=None, delta_bias=None,
                z=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """Enqueue the forward on ``stream`` (default: torch's current stream).

        delta_bias ([D] float32) and z ([B, L, D], plan dtype) select the fused
        prologue / epilogue (``sscan_forward_gated``)."""
        Bt, L, D, N = self.shape
        if y is None:
            y = torch.empty((Bt, L, D), dtype=self.dtype, device=u.device)
        if h_final is None and want_final:
            h_final = torch.empty((Bt, D, N), dtype=torch.float32, device=u.device)
        for name, t, shape, dt in (("u", u, (Bt, L, D), self.dtype),
                                   ("delta", delta, (Bt, L, D), self.dtype),
                                   ("A", A, (D, N), torch.float32),
                                   ("B", B, (Bt, L, N), self.dtype),
                                   ("C", C, (Bt, L, N), self.dtype),
                                   ("h0", h0, (Bt, D, N), torch.float32),
                                   ("y", y, (Bt, L, D), self.dtype),
                                   ("h_final", h_final, (Bt, D, N), torch.float32),
                                   ("delta_bias", delta_bias, (D,), torch.float32),
                                   ("z", z, (Bt, L, D), self.dtype)):
            if t is None:
                continue
            if tuple(t.shape) != shape or t.dtype != dt or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name}: want contiguous CUDA {dt} {shape}, got "
                                 f"{t.dtype} {tuple(t.shape)} on {t.device}")
        if workspace is None and self.workspace_bytes:
            workspace = self.new_workspace(u.device)
        if stream is None:
            stream = torch.cuda.current_stream(u.device)
        if delta_bias is None and z is None:
            rc = lib().sscan_forward(self._h, _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                                     _ptr(h0), _ptr(y), _ptr(h_final), _ptr(workspace),
                                     ctypes.c_void_p(stream.cuda_stream))
            what = "sscan_forward"
        else:
            rc = lib().sscan_forward_gated(self._h, _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                                           _ptr(h0), _ptr(delta_bias), _ptr(z), _ptr(y), _ptr(h_final),
                                           _ptr(workspace), ctypes.c_void_p(stream.cuda_stream))
            what = "sscan_forward_gated"
        if rc != OK:
            raise SscanError(rc, what)
        return y, h_final

    def host_workspace_bytes(self) -> int:
        n = int(lib().sscan_host_workspace_bytes(self._h))
        if n == 0:
            raise SscanError(ERR_INVALID, "sscan_host_workspace_bytes")
        return n

    def forward_host(self, u, delta, A, B, C, h0, y, h_final, delta_bias=None, z=None, stream=None,
                     workspace=None):
        """Enqueue ``sscan_forward_host`` on ``stream``: every tensor a contiguous CPU
        tensor (pinned for overlapped copies), the device workspace allocated here
        unless given.  Returns without waiting; synchronise ``stream`` before
        reading y and h_final."""
        Bt, L, D, N = self.shape
        for name, t, shape, dt in (("u", u, (Bt, L, D), self.dtype),
                                   ("delta", delta, (Bt, L, D), self.dtype),
                                   ("A", A, (D, N), torch.float32),
                                   ("B", B, (Bt, L, N), self.dtype),
                                   ("C", C, (Bt, L, N), self.dtype),
                                   ("h0", h0, (Bt, D, N), torch.float32),
                                   ("y", y, (Bt, L, D), self.dtype),
                                   ("h_final", h_final, (Bt, D, N), torch.float32),
                                   ("delta_bias", delta_bias, (D,), torch.float32),
                                   ("z", z, (Bt, L, D), self.dtype)):
            if t is None:
                continue
            if tuple(t.shape) != shape or t.dtype != dt or t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name}: want contiguous host {dt} {shape}, got "
                                 f"{t.dtype} {tuple(t.shape)} on {t.device}")
        if stream is None:
            stream = torch.cuda.current_stream()
        if workspace is None:
            workspace = torch.empty(self.host_workspace_bytes(), dtype=torch.uint8, device=stream.device)
        rc = lib().sscan_forward_host(self._h, _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0),
                                      _ptr(delta_bias), _ptr(z), _ptr(y), _ptr(h_final), _ptr(workspace),
                                      ctypes.c_void_p(stream.cuda_stream))
        if rc != OK:
            raise SscanError(rc, "sscan_forward_host")
        workspace.record_stream(stream)
        return y, h_final

    def backward(self, u, delta, A, B, C, h0, dy, dh_final=None, want_dh0: bool = True, stream=None,
                 delta_bias=None, z=None) -> dict:
        """Gradients of this plan's forward: returns a dict with du, ddelta (plan dtype), dA,
        dB, dC and dh0 (fp32) given dy (and optionally dh_final); with delta_bias and z
        (the fused layer, ``sscan_backward_gated``) also ddelta_bias (fp32) and dz."""
        Bt, L, D, N = self.shape
        dev = u.device
        out = {"du": torch.empty((Bt, L, D), dtype=self.dtype, device=dev),
               "ddelta": torch.empty((Bt, L, D), dtype=self.dtype, device=dev),
               "dA": torch.empty((D, N), dtype=torch.float32, device=dev),
               "dB": torch.empty((Bt, L, N), dtype=torch.float32, device=dev),
               "dC": torch.empty((Bt, L, N), dtype=torch.float32, device=dev),
               "dh0": torch.empty((Bt, D, N), dtype=torch.float32, device=dev) if want_dh0 else None,
               "ddelta_bias": torch.empty((D,), dtype=torch.float32, device=dev) if delta_bias is not None else None,
               "dz": torch.empty((Bt, L, D), dtype=self.dtype, device=dev) if z is not None else None}
        wsb = int(lib().sscan_backward_workspace_bytes(Bt, L, D, N))
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        flags = (ZOH if self.zoh else 0) | (DELTA_SOFTPLUS if self.delta_softplus else 0)
        rc = lib().sscan_backward_gated(Bt, L, D, N, _dtype_code(self.dtype), flags,
                                        _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0),
                                        _ptr(delta_bias), _ptr(z), _ptr(dy), _ptr(dh_final), _ptr(out["du"]),
                                        _ptr(out["ddelta"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]),
                                        _ptr(out["dh0"]), _ptr(out["ddelta_bias"]), _ptr(out["dz"]), _ptr(ws),
                                        ctypes.c_void_p(stream.cuda_stream))
        if rc != OK:
            raise SscanError(rc, "sscan_backward_gated")
        return out

    def status(self, stream=None) -> int:
        """Synchronise ``stream`` and read (and clear) the plan's device status word."""
        if stream is None:
            stream = torch.cuda.current_stream()
        return int(lib().sscan_get_status(self._h, ctypes.c_void_p(stream.cuda_stream)))


_plans: dict = {}


def get_plan(B, L, D, N, dtype=torch.float32, zoh=False, delta_softplus=False) -> Plan:
    key = (int(B), int(L), int(D), int(N), dtype, bool(zoh), bool(delta_softplus),
           torch.cuda.current_device())
    p = _plans.get(key)
    if p is None:
        p = _plans[key] = Plan(B, L, D, N, dtype, zoh, delta_softplus)
    return p


def forward(u, delta, A, B, C, h0=None, zoh: bool = False, want_final: bool = True,
            delta_bias=None, delta_softplus: bool = False, z=None):
    """Selective-scan forward on CUDA tensors: returns (y [B,L,D], h_final [B,D,N] or None).

    u, delta: [B, L, D] float32 or bfloat16; A: [D, N] float32; B, C: [B, L, N]
    (dtype of u); h0: [B, D, N] float32 or None.  Fused prologue / epilogue:
    delta_bias [D] float32 and delta_softplus (delta <- softplus(delta + bias)),
    z [B, L, D] (dtype of u; y <- y * silu(z)).
    """
    Bt, L, D = u.shape
    N = A.shape[1]
    return get_plan(Bt, L, D, N, u.dtype, zoh, delta_softplus).forward(
        u, delta, A, B, C, h0, want_final=want_final, delta_bias=delta_bias, z=z)


def forward_host(u, delta, A, B, C, h0=None, zoh: bool = False, device="cuda", out=None,
                 delta_bias=None, delta_softplus: bool = False, z=None, stream=None):
    """Forward on host (CPU) tensors through ``sscan_forward_host``: the library
    copies the inputs to the device piece by piece, scans, and copies y and
    h_final back, the copies of neighbouring pieces overlapping the scan.
    Page-locked (pinned) host tensors let the copies run asynchronously;
    ``out`` = (y_host, h_final_host) reuses output buffers; delta_bias,
    delta_softplus and z select the fused prologue / epilogue.  Waits for the
    stream before returning.  Returns (y_host, h_final_host)."""
    dev = torch.device(device)
    Bt, L, D = u.shape
    N = A.shape[1]
    plan = get_plan(Bt, L, D, N, u.dtype, zoh, delta_softplus)
    if out is None:
        pin = u.is_pinned()
        out = (torch.empty((Bt, L, D), dtype=u.dtype, pin_memory=pin),
               torch.empty((Bt, D, N), dtype=torch.float32, pin_memory=pin))
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    plan.forward_host(u, delta, A, B, C, h0, out[0], out[1], delta_bias=delta_bias, z=z, stream=stream)
    stream.synchronize()
    return out


def ssd_forward(x, delta, A, B, C, h0=None, y=None, h_final=None, want_final: bool = True,
                status=None, stream=None):
    """Mamba-2 SSD forward (``sscan_ssd_forward``) on CUDA tensors.

    x: [B, L, H, P] bfloat16; delta: [B, L, H] float32; A: [H] float32; B, C:
    [B, L, N] bfloat16; h0: [B, H, N, P] float32 or None; status: a CUDA int32
    tensor of one element the kernel ORs error bits into, or None.
    Returns (y [B, L, H, P] bfloat16, h_final [B, H, N, P] float32 or None)."""
    Bt, L, H, P = x.shape
    N = B.shape[-1]
    dev = x.device
    if y is None:
        y = torch.empty((Bt, L, H, P), dtype=torch.bfloat16, device=dev)
    if h_final is None and want_final:
        h_final = torch.empty((Bt, H, N, P), dtype=torch.float32, device=dev)
    for name, t, shape, dt in (("x", x, (Bt, L, H, P), torch.bfloat16), ("delta", delta, (Bt, L, H), torch.float32),
                               ("A", A, (H,), torch.float32), ("B", B, (Bt, L, N), torch.bfloat16),
                               ("C", C, (Bt, L, N), torch.bfloat16), ("h0", h0, (Bt, H, N, P), torch.float32),
                               ("y", y, (Bt, L, H, P), torch.bfloat16),
                               ("h_final", h_final, (Bt, H, N, P), torch.float32),
                               ("status", status, (1,), torch.int32)):
        if t is None:
            continue
        if tuple(t.shape) != shape or t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: want contiguous CUDA {dt} {shape}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    rc = lib().sscan_ssd_forward(Bt, L, H, P, N, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0),
                                 _ptr(y), _ptr(h_final), _ptr(status), ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise SscanError(rc, "sscan_ssd_forward")
    return y, h_final


# --------------------------------------------------------------------------
# Recurrent block operators: the gated linear recurrence and the layer norm.  A decode
# step runs in a few microseconds on the device, so these wrappers keep to what a call
# needs: checks of attributes (written out: a function call each would cost as much as the
# check), one allocation per output, the current stream's handle.  None of them records an
# autograd graph: outputs never require a gradient, and the backward functions are called by hand.

_F32 = torch.float32
_CODES = {torch.float32: F32, torch.bfloat16: BF16}
# torch's quicker names for these are private: the public ones where it lacks them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _unlike(name, t, shape, dt, d):
    """The error of a tensor that is not a contiguous one of this shape, dtype and device."""
    return ValueError(f"{name}: want contiguous {dt} {tuple(shape)} on cuda:{d}, got {t.dtype} {tuple(t.shape)} "
                      f"on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _elsewhere(fn, ref, stream, args):
    """fn(stream handle, *args) where the call is not simply on ref's current device and
    stream: with ref's device current, and new tensors allocated on the call's stream, so
    that the allocator knows who uses them."""
    if not ref.is_cuda:
        raise ValueError(f"want CUDA tensors, got one on {ref.device}")
    dev = ref.device
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"stream on {stream.device}, tensors on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return fn(stream.cuda_stream, *args)


def _adr(t):
    return None if t is None else t.data_ptr()


def _workspace(given, nbytes, like):
    if given is None:
        return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    if given.dtype != torch.uint8 or given.device != like.device or not given.is_contiguous() or given.numel() < nbytes:
        raise ValueError(f"workspace: want at least {nbytes} contiguous uint8 on {like.device}, got {given.dtype} "
                         f"{tuple(given.shape)} on {given.device}")
    return given


@functools.lru_cache(maxsize=1024)
def _glr_sizes(B: int, L: int, D: int):
    """(values of the saved states, bytes of the backward pass's workspace) of a shape"""
    return (int(lib().sscan_glr_states_bytes(B, L, D)) // 4, int(lib().sscan_glr_backward_workspace_bytes(B, L, D)))


def new_glr_states(B: int, L: int, D: int, device="cuda") -> torch.Tensor:
    """A buffer for the states that ``glr_forward`` saves for ``glr_backward``."""
    return torch.empty(_glr_sizes(B, L, D)[0], dtype=_F32, device=device)


_ALL_TRIES = 2 ** 32 - 1  # the library's own limit of a wait


def _check_status(status, d):
    if status.shape != (1,) or status.dtype != torch.int32 or status.get_device() != d:
        raise _unlike("status", status, (1,), torch.int32, d)


def glr_forward(x, gate, rate=None, input_gate=None, h0=None, y=None, h_final=None, want_final: bool = True,
                states=None, want_states: bool = False, stream=None, status=None):
    """Gated linear recurrence (``sscan_glr_forward``) on CUDA tensors.

    x, gate and input_gate (or None): [B, L, D] float32 or bfloat16; rate: [D] float32 > 0
    (above 2^21: as 2^21) or None; h0: [B, D] float32 or None.  h_final may be h0 (a decode step in place).
    ``want_states`` returns the saved states that ``glr_backward`` reads (or pass a buffer
    of ``new_glr_states`` as ``states``).  Work and new tensors are on ``stream`` (default:
    the current stream of x's device).  ``status``: a CUDA int32 tensor of one element, set to
    non-zero when a wait inside the kernel gives up (outputs then hold NaN), or None.
    Returns (y [B, L, D], h_final [B, D] float32 or None, states or None)."""
    d = x.get_device()
    if stream is None and d >= 0 and d == _device_now():
        return _glr_forward(_raw_stream(d), x, gate, rate, input_gate, h0, y, h_final, want_final, states, want_states,
                            status)
    return _elsewhere(_glr_forward, x, stream,
                      (x, gate, rate, input_gate, h0, y, h_final, want_final, states, want_states, status))


def _glr_forward(st, x, gate, rate, input_gate, h0, y, h_final, want_final, states, want_states, status):
    shape, dt, d = x.shape, x.dtype, x.get_device()
    code = _CODES.get(dt)
    if code is None:
        _dtype_code(dt)  # raises
    if len(shape) != 3:
        raise ValueError(f"x: want [B, L, D], got {tuple(shape)}")
    B, L, D = shape
    if not x.is_contiguous():
        raise _unlike("x", x, shape, dt, d)
    if gate.shape != shape or gate.dtype != dt or gate.get_device() != d or not gate.is_contiguous():
        raise _unlike("gate", gate, shape, dt, d)
    if input_gate is not None:
        if (input_gate.shape != shape or input_gate.dtype != dt or input_gate.get_device() != d
                or not input_gate.is_contiguous()):
            raise _unlike("input_gate", input_gate, shape, dt, d)
    if rate is not None:
        if rate.shape != (D,) or rate.dtype != _F32 or rate.get_device() != d or not rate.is_contiguous():
            raise _unlike("rate", rate, (D,), _F32, d)
    if h0 is not None:
        if h0.shape != (B, D) or h0.dtype != _F32 or h0.get_device() != d or not h0.is_contiguous():
            raise _unlike("h0", h0, (B, D), _F32, d)
    if y is None:
        y = torch.empty_like(x)
    else:
        if y.shape != shape or y.dtype != dt or y.get_device() != d or not y.is_contiguous():
            raise _unlike("y", y, shape, dt, d)
    if h_final is not None:
        if h_final.shape != (B, D) or h_final.dtype != _F32 or h_final.get_device() != d or not h_final.is_contiguous():
            raise _unlike("h_final", h_final, (B, D), _F32, d)
    elif want_final:
        h_final = x.new_empty((B, D), dtype=_F32) if h0 is None else torch.empty_like(h0)
    if states is not None:
        if (states.shape != (_glr_sizes(B, L, D)[0],) or states.dtype != _F32 or states.get_device() != d
                or not states.is_contiguous()):
            raise _unlike("states", states, (_glr_sizes(B, L, D)[0],), _F32, d)
    elif want_states:
        states = x.new_empty(_glr_sizes(B, L, D)[0], dtype=_F32)
    if status is None:
        rc = (_lib or lib()).sscan_glr_forward(
            B, L, D, code, x.data_ptr(), gate.data_ptr(), _adr(input_gate), _adr(rate), _adr(h0), y.data_ptr(),
            _adr(h_final), _adr(states), st)
    else:
        _check_status(status, d)
        rc = (_lib or lib()).sscan_glr_forward_checked(
            B, L, D, code, x.data_ptr(), gate.data_ptr(), _adr(input_gate), _adr(rate), _adr(h0), y.data_ptr(),
            _adr(h_final), _adr(states), status.data_ptr(), _ALL_TRIES, st)
    if rc != OK:
        raise SscanError(rc, "sscan_glr_forward")
    return y, h_final, states


def glr_backward(x, gate, dy, states, rate=None, input_gate=None, dh_final=None, want_dh0: bool = True,
                 workspace=None, stream=None, status=None) -> dict:
    """Gradients of ``glr_forward`` (``sscan_glr_backward``): x, gate, rate and input_gate as
    passed to it, ``states`` as it returned them, dy [B, L, D] and dh_final [B, D] float32
    (or None).  Returns a dict with dx, dgate and dinput_gate (dtype of x; the last None
    without an input gate), drate ([D] float32, None without a rate) and dh0 ([B, D]
    float32, None unless wanted).  ``workspace``: a CUDA uint8 tensor of at least
    ``sscan_glr_backward_workspace_bytes`` (default: allocated here).  ``status`` as for
    ``glr_forward``."""
    d = x.get_device()
    if stream is None and d >= 0 and d == _device_now():
        return _glr_backward(_raw_stream(d), x, gate, dy, states, rate, input_gate, dh_final, want_dh0, workspace,
                             status)
    return _elsewhere(_glr_backward, x, stream,
                      (x, gate, dy, states, rate, input_gate, dh_final, want_dh0, workspace, status))


def _glr_backward(st, x, gate, dy, states, rate, input_gate, dh_final, want_dh0, workspace, status):
    shape, dt, d = x.shape, x.dtype, x.get_device()
    code = _CODES.get(dt)
    if code is None:
        _dtype_code(dt)  # raises
    if len(shape) != 3:
        raise ValueError(f"x: want [B, L, D], got {tuple(shape)}")
    B, L, D = shape
    if not x.is_contiguous():
        raise _unlike("x", x, shape, dt, d)
    if gate.shape != shape or gate.dtype != dt or gate.get_device() != d or not gate.is_contiguous():
        raise _unlike("gate", gate, shape, dt, d)
    if dy.shape != shape or dy.dtype != dt or dy.get_device() != d or not dy.is_contiguous():
        raise _unlike("dy", dy, shape, dt, d)
    n_states, n_workspace = _glr_sizes(B, L, D)
    if states.shape != (n_states,) or states.dtype != _F32 or states.get_device() != d or not states.is_contiguous():
        raise _unlike("states", states, (n_states,), _F32, d)
    dig = drate = dh0 = None
    if input_gate is not None:
        if (input_gate.shape != shape or input_gate.dtype != dt or input_gate.get_device() != d
                or not input_gate.is_contiguous()):
            raise _unlike("input_gate", input_gate, shape, dt, d)
        dig = torch.empty_like(x)
    if dh_final is not None:
        if (dh_final.shape != (B, D) or dh_final.dtype != _F32 or dh_final.get_device() != d
                or not dh_final.is_contiguous()):
            raise _unlike("dh_final", dh_final, (B, D), _F32, d)
    if want_dh0:
        dh0 = x.new_empty((B, D), dtype=_F32) if dh_final is None else torch.empty_like(dh_final)
    if rate is not None:
        if rate.shape != (D,) or rate.dtype != _F32 or rate.get_device() != d or not rate.is_contiguous():
            raise _unlike("rate", rate, (D,), _F32, d)
        drate = torch.empty_like(rate)
        workspace = _workspace(workspace, n_workspace, x)
    else:
        workspace = None
    dx, dgate = torch.empty_like(x), torch.empty_like(x)
    if status is None:
        rc = (_lib or lib()).sscan_glr_backward(
            B, L, D, code, x.data_ptr(), gate.data_ptr(), _adr(input_gate), _adr(rate), states.data_ptr(), dy.data_ptr(),
            _adr(dh_final), dx.data_ptr(), dgate.data_ptr(), _adr(dig), _adr(drate), _adr(dh0), _adr(workspace), st)
    else:
        _check_status(status, d)
        rc = (_lib or lib()).sscan_glr_backward_checked(
            B, L, D, code, x.data_ptr(), gate.data_ptr(), _adr(input_gate), _adr(rate), states.data_ptr(), dy.data_ptr(),
            _adr(dh_final), dx.data_ptr(), dgate.data_ptr(), _adr(dig), _adr(drate), _adr(dh0), _adr(workspace),
            status.data_ptr(), _ALL_TRIES, st)
    if rc != OK:
        raise SscanError(rc, "sscan_glr_backward")
    return {"dx": dx, "dgate": dgate, "dinput_gate": dig, "drate": drate, "dh0": dh0}


def _norm_types(x_dt, r_dt):
    """(dtype code, residual flag) of a norm whose x and residual have these dtypes."""
    code = _CODES.get(x_dt)
    if code is None:
        _dtype_code(x_dt)  # raises
    if r_dt == x_dt:
        return code, 0
    if r_dt == _F32:
        return code, NORM_RESIDUAL_F32
    raise TypeError(f"residual of {r_dt} with x of {x_dt} (the same, or float32)")


def norm_forward(x, weight=None, bias=None, residual=None, eps: float = 1e-5, rms: bool = False,
                 want_stats: bool = True, stream=None):
    """Layer norm over the last axis (``sscan_norm_forward``) on CUDA tensors, after the
    residual addition when ``residual`` is given.

    x: [..., D] float32 or bfloat16; residual: the shape of x, its dtype or float32;
    weight, bias: [D] float32 or None; ``rms`` removes no mean.  Returns (y, s, mean, rstd):
    y in x's dtype; s = x + residual in the residual's dtype (x itself without a residual);
    mean and rstd float32, one per row (mean None with rms, both None unless
    ``want_stats``).  Work and new tensors are on ``stream`` (default: the current stream
    of x's device)."""
    d = x.get_device()
    if stream is None and d >= 0 and d == _device_now():
        return _norm_forward(_raw_stream(d), x, weight, bias, residual, eps, rms, want_stats)
    return _elsewhere(_norm_forward, x, stream, (x, weight, bias, residual, eps, rms, want_stats))


def _norm_forward(st, x, weight, bias, residual, eps, rms, want_stats):
    shape, dt, d = x.shape, x.dtype, x.get_device()
    if len(shape) < 1:
        raise ValueError("x: want [..., D]")
    D = shape[-1]
    if not x.is_contiguous():
        raise _unlike("x", x, shape, dt, d)
    if residual is None:
        code, flags = _norm_types(dt, dt)
        s = x
    else:
        code, flags = _norm_types(dt, residual.dtype)
        if residual.shape != shape or residual.get_device() != d or not residual.is_contiguous():
            raise _unlike("residual", residual, shape, residual.dtype, d)
        s = torch.empty_like(residual)
    if weight is not None:
        if weight.shape != (D,) or weight.dtype != _F32 or weight.get_device() != d or not weight.is_contiguous():
            raise _unlike("weight", weight, (D,), _F32, d)
    if bias is not None:
        if bias.shape != (D,) or bias.dtype != _F32 or bias.get_device() != d or not bias.is_contiguous():
            raise _unlike("bias", bias, (D,), _F32, d)
    y = torch.empty_like(x)
    rows = x.numel() // D if D else shape[:-1].numel()
    mean = rstd = None
    if want_stats:
        rstd = x.new_empty(shape[:-1], dtype=_F32)
        mean = None if rms else torch.empty_like(rstd)
    rc = (_lib or lib()).sscan_norm_forward(
        rows, D, code, flags | (NORM_RMS if rms else 0), eps, x.data_ptr(), _adr(residual), _adr(weight), _adr(bias),
        y.data_ptr(), None if residual is None else s.data_ptr(), _adr(mean), _adr(rstd), st)
    if rc != OK:
        raise SscanError(rc, "sscan_norm_forward")
    return y, s, mean, rstd


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows: int, D: int) -> int:
    return int(lib().sscan_norm_backward_workspace_bytes(rows, D))


def norm_backward(dy, s, mean, rstd, weight=None, dresidual=None, rms: bool = False, want_dweight: bool = True,
                  want_dbias: bool = False, workspace=None, stream=None) -> dict:
    """Gradients of ``norm_forward`` (``sscan_norm_backward``): dy [..., D] in the forward's
    dtype of x; s, mean, rstd as it returned them; weight as passed to it; dresidual the
    gradient that reaches s from its other uses (dtype of s) or None.  Returns a dict with
    dx (dtype of dy), dresidual (dtype of s; the same tensor as dx where the types are
    equal), dweight and dbias ([D] float32 or None).  ``workspace``: a CUDA uint8 tensor of
    at least ``sscan_norm_backward_workspace_bytes`` (default: allocated here)."""
    d = dy.get_device()
    if stream is None and d >= 0 and d == _device_now():
        return _norm_backward(_raw_stream(d), dy, s, mean, rstd, weight, dresidual, rms, want_dweight, want_dbias,
                              workspace)
    return _elsewhere(_norm_backward, dy, stream,
                      (dy, s, mean, rstd, weight, dresidual, rms, want_dweight, want_dbias, workspace))


def _norm_backward(st, dy, s, mean, rstd, weight, dresidual, rms, want_dweight, want_dbias, workspace):
    shape, dt, d = dy.shape, dy.dtype, dy.get_device()
    if len(shape) < 1:
        raise ValueError("dy: want [..., D]")
    D, row_shape = shape[-1], shape[:-1]
    code, flags = _norm_types(dt, s.dtype)
    if not dy.is_contiguous():
        raise _unlike("dy", dy, shape, dt, d)
    if s.shape != shape or s.get_device() != d or not s.is_contiguous():
        raise _unlike("s", s, shape, s.dtype, d)
    if rstd.shape != row_shape or rstd.dtype != _F32 or rstd.get_device() != d or not rstd.is_contiguous():
        raise _unlike("rstd", rstd, row_shape, _F32, d)
    if not rms:
        if mean is None:
            raise ValueError("mean: wanted without rms")
        if mean.shape != row_shape or mean.dtype != _F32 or mean.get_device() != d or not mean.is_contiguous():
            raise _unlike("mean", mean, row_shape, _F32, d)
    elif mean is not None:
        raise ValueError("mean: must be None with rms")
    dweight = dbias = None
    if weight is not None:
        if weight.shape != (D,) or weight.dtype != _F32 or weight.get_device() != d or not weight.is_contiguous():
            raise _unlike("weight", weight, (D,), _F32, d)
        if want_dweight:
            dweight = torch.empty_like(weight)
    if dresidual is not None:
        if (dresidual.shape != shape or dresidual.dtype != s.dtype or dresidual.get_device() != d
                or not dresidual.is_contiguous()):
            raise _unlike("dresidual", dresidual, shape, s.dtype, d)
    rows = row_shape.numel()
    ds = torch.empty_like(s)
    dx = torch.empty_like(dy) if s.dtype != dt else None
    if want_dbias:
        dbias = dy.new_empty((D,), dtype=_F32) if weight is None else torch.empty_like(weight)
    if dweight is not None or dbias is not None:
        workspace = _workspace(workspace, _norm_workspace(rows, D), dy)
    else:
        workspace = None
    rc = (_lib or lib()).sscan_norm_backward(
        rows, D, code, flags | (NORM_RMS if rms else 0), dy.data_ptr(), s.data_ptr(), _adr(mean), rstd.data_ptr(),
        _adr(weight), _adr(dresidual), ds.data_ptr(), _adr(dx), _adr(dweight), _adr(dbias), _adr(workspace), st)
    if rc != OK:
        raise SscanError(rc, "sscan_norm_backward")
    return {"dx": ds if dx is None else dx, "dresidual": ds, "dweight": dweight, "dbias": dbias}
