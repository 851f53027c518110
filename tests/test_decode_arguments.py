"""What a DecodeAttention refuses, and that a refusal leaves it as it was."""
import pytest
import torch

import int8_quantized_gb300 as q
from int8_quantized_gb300 import decode


@pytest.mark.parametrize("kw", [dict(budget=24), dict(sink=-1), dict(recent=-1), dict(sink=40, recent=25),
                                dict(budget=0), dict(budget=96)])
def test_a_layer_refuses_what_eviction_would(kw):
    args = dict(sequences=1, q_heads=4, kv_heads=2, head_dim=64, capacity=96, budget=64)
    args.update(kw)
    with pytest.raises(ValueError, match="budget"):
        decode.DecodeAttention(None, None, None, None, None, None, **args)


def state(layer):
    return (list(layer.free), [list(o) for o in layer.owned], list(layer.length), list(layer.position),
            layer.table.tolist(), layer.cache.k.clone(), layer.cache.score.clone())


def same(a, b):
    return a[:5] == b[:5] and torch.equal(a[5], b[5]) and torch.equal(a[6], b[6])


@pytest.mark.gpu
def test_a_refused_eviction_keeps_the_pages(dev):
    layer = decode.random_layer(sequences=2, hidden=128, q_heads=4, kv_heads=2, head_dim=64, capacity=20, budget=12,
                                sink=2, recent=3)
    assert (layer.sink, layer.recent) == (2, 3)
    x = torch.randn((2, 128), device=dev).to(torch.bfloat16)
    out = torch.empty_like(x)
    for _ in range(20):
        layer.step(x, out)
    layer.recent = 11
    before = state(layer)
    with pytest.raises(q.I8QError):
        layer.evict(1)
    assert same(state(layer), before)
    with pytest.raises(q.I8QError):
        layer.step(x, out)
    assert same(state(layer), before)
    layer.recent = 3
    layer.step(x, out)
    assert layer.length == [13, 13]
    q.sync_status()


@pytest.mark.gpu
def test_a_step_past_the_last_position_is_refused(dev):
    layer = decode.random_layer(sequences=2, hidden=128, q_heads=4, kv_heads=2, head_dim=64, positions=17)
    x = torch.randn((2, 128), device=dev).to(torch.bfloat16)
    out = torch.empty_like(x)
    for _ in range(17):
        layer.step(x, out)
    before = state(layer)
    with pytest.raises(ValueError, match="position"):
        layer.step(x, out)
    assert same(state(layer), before)
    q.sync_status()
