"""Tensors on another device than the current one, on which the kernels would
run, are refused on the host."""
import pytest
import torch

import int8_quantized_gb300 as q
from test_binding_arguments import on


@pytest.fixture
def second(monkeypatch):
    class Library:
        def __getattr__(self, name):
            raise AssertionError("the library was called")

    monkeypatch.setattr(q, "_L", lambda: Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lambda t: on(t, torch.device("cuda:1"))


def test_sample(second):
    x = second(torch.zeros((2, 50)))
    u, t = second(torch.zeros(2)), second(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="not the current device"):
        q.sample(x, u, t)


def test_matmul_nbits(second):
    B, s = second(torch.zeros((16, 2, 16), dtype=torch.uint8)), second(torch.zeros((16, 2)))
    with pytest.raises(ValueError, match="not the current device"):
        q.MatMulNBits(B, s, 64, 32)
    with pytest.raises(ValueError, match="one device"):
        q.MatMulNBits(B, on(torch.zeros((16, 2)), torch.device("cuda:0")), 64, 32)


def test_sample_settings_beside_the_logits(second, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    x, t = second(torch.zeros((2, 50))), second(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="temperature must be"):
        q.sample(x, second(torch.zeros(2)), t, temperature=on(torch.zeros(2), torch.device("cuda:0")))


@pytest.mark.parametrize("name", ["q_norm", "k_norm"])
def test_norms_of_the_heads(second, monkeypatch, name):
    cache = type("Cache", (), {"_ref": None, "shape": (1, 1, 16, 64)})()
    i, x, w = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1, 64)), torch.ones(64)

    def call(place, norm):
        to = lambda t: on(t, torch.device(place))
        q.kv_append(cache, to(torch.zeros((1, 1), dtype=torch.int32)), to(i), to(i), to(x), to(x), q=to(x), q_out=to(x.clone()),
                    **{name: norm})

    with pytest.raises(TypeError, match=f"{name} must be a tensor beside k"):
        call("cuda:0", second(w))
    with pytest.raises(ValueError, match="not the current device"):
        call("cuda:1", second(w))
    with pytest.raises(AssertionError, match="the library was called"):
        call("cuda:0", on(w, torch.device("cuda:0")))
