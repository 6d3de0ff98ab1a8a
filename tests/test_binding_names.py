"""The block operators' binding without torch's private names for the current stream and device."""
import importlib.util

import pytest
import torch

from selective_state_space_32_b200 import sscan as S


@pytest.fixture
def without(monkeypatch):
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("sscan_without_private_names", S.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.undo()   # torch itself calls them
    return m


def test_there_is_another_way(without, monkeypatch):
    assert without._device_now is torch.cuda.current_device
    stream = type("Stream", (), {"cuda_stream": 77})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: stream if d == 3 else None)
    assert without._raw_stream(3) == 77


@pytest.mark.gpu
def test_calls_give_the_same(without):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_32_b200 import build
    build.build()
    x, gate = torch.randn(2, 30, 64, device="cuda"), torch.randn(2, 30, 64, device="cuda")
    out = []
    for m in (S, without):
        y, hf, st = m.glr_forward(x, gate, want_states=True)
        g = m.glr_backward(x, gate, x, st)
        n = m.norm_forward(x)
        b = m.norm_backward(x, n[1], n[2], n[3])
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            y2 = m.glr_forward(x, gate)[0]
            torch.cuda.current_stream().synchronize()
        out.append([y, hf, g["dx"], g["dgate"], n[0], b["dx"], y2])
    assert all(torch.equal(p, q) for p, q in zip(*out))
