"""What the binding itself checks, on the host."""
import pytest
import torch

import int8_quantized_gb300 as q


def test_the_current_stream_initialises_cuda(monkeypatch):
    """Where CUDA cannot be initialised (a forked child, no driver) the call
    says what torch says, for every operator."""
    def refuse():
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")

    monkeypatch.setattr(torch.cuda, "_lazy_init", refuse)
    for call in (q._stream, q.sync_status, lambda: q.measure_int8_mma_peak(1)):
        with pytest.raises(RuntimeError, match="re-initialize CUDA"):
            call()


def test_a_torch_without_cuda_says_so(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)

    def refuse():
        raise AssertionError("Torch not compiled with CUDA enabled")

    monkeypatch.setattr(torch.cuda, "_lazy_init", refuse)
    with pytest.raises(AssertionError, match="not compiled with CUDA"):
        q._stream()
