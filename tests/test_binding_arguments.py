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


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lies on a GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: self.where)


def on(t, where="cuda:0"):
    t = t.as_subclass(OnDevice)
    t.where = where
    return t


def pool(shape, dtype=torch.int8, where="cuda:0"):
    return on(torch.zeros(shape, dtype=dtype), where)


def test_cache_pools_lie_on_one_device():
    shape = (2, 2, 16, 64)
    scales = [pool(shape[:3], torch.float32) for _ in range(2)]
    q.KVCache(pool(shape), pool(shape), *scales)
    with pytest.raises(TypeError, match="v must be"):
        q.KVCache(pool(shape), pool(shape, where="cuda:1"), *scales)
    with pytest.raises(TypeError, match="v_scale must be"):
        q.KVCache(pool(shape), pool(shape), scales[0], pool(shape[:3], torch.float32, "cuda:1"))
