"""The stream that the binding launches on when none is given."""
import pytest
import torch

from gpu_util import cuda_ok

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")


@pytest.mark.parametrize("name", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_a_torch_without_the_raw_functions(monkeypatch, name):
    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 77, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    assert mhc._stream(None) == 77
    monkeypatch.delattr(torch._C, name)
    assert mhc._stream(None) == 1234


@pytest.mark.gpu
@pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")
def test_it_is_the_current_stream():
    assert mhc._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert mhc._stream(None) == side.cuda_stream
