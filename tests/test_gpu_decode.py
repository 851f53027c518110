"""The decoder attention layer that runs the cache operators together: each
step against a plain form over what the cache holds, across evictions."""
import numpy as np
import pytest
import torch

import int8_quantized_gb300 as q
from int8_quantized_gb300 import decode
from test_gpu_kv_cache import host, reference_attention, reference_kept, rotate

pytestmark = pytest.mark.gpu


def test_decode_steps_match_the_plain_form(dev):
    layer = decode.random_layer(sequences=3, hidden=256, q_heads=8, kv_heads=2, head_dim=64, capacity=40, budget=24,
                                seed=1)
    layer.sink, layer.recent = 2, 6
    g = torch.Generator()
    g.manual_seed(5)
    out = torch.empty((3, 256), dtype=torch.bfloat16, device=dev)
    evicted = []
    plain = layer.evict

    def watched(b):
        before, n = host(layer.cache.score), layer.length[b]
        row = layer.table[b].cpu().numpy()
        t = np.arange(n)
        score = before[row[t // layer.page], :, t % layer.page].astype(np.float32)
        kept = plain(b)
        for h in range(layer.H):
            assert np.array_equal(kept[h].cpu().numpy(),
                                  reference_kept(score[:, h], n, layer.budget, layer.sink, layer.recent))
        evicted.append((b, n))
        return kept

    layer.evict = watched
    layer.length[0] = 0
    for step in range(75):
        x = torch.randn((3, 256), generator=g).to(torch.bfloat16).to(dev)
        layer.step(x, out)
        # the step's keys as the cache must hold them: half a step of the row's scale, and bf16 projections
        rows = layer.qkv.view(3, 12, 64)
        key, value = rows[:, 8:10].float().cpu().numpy(), rows[:, 10:].float().cpu().numpy()
        pos = np.full((1, 3), step)
        key = rotate(key, pos, layer.cos.cpu().numpy(), layer.sin.cpu().numpy(), None, False)
        tab = layer.table.cpu().numpy()
        for b in range(3):
            t = layer.length[b] - 1
            pg, off = tab[b, t // layer.page], t % layer.page
            for pool, scale, want in ((layer.cache.k, layer.cache.k_scale, key), (layer.cache.v, layer.cache.v_scale, value)):
                s = host(scale[pg, :, off])[:, None]
                got = host(pool[pg, :, off]) * s
                assert np.all(np.abs(got - want[b]) <= 0.501 * s)
        # the step's attention over what the cache holds: q was turned in place
        ref, *_ = reference_attention(layer.cache, layer.table, layer.length, rows[:, :8], 0, 64 ** -0.5)
        got = host(layer.attended)
        # weights of 16 bits, a bf16 output, and scores that move by 2^-20 of sum |q k|
        assert np.abs(got - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4
        again = torch.empty_like(out)
        layer.out_gemm.forward(layer.attended.view(3, -1), again)
        assert torch.equal(out, again)
    q.sync_status()
    # full at 40, cut to 24, then every 16 tokens
    assert evicted == [(b, 40) for _ in range(3) for b in range(3)]
    assert layer.length == [27] * 3 and layer.position == [75] * 3
    assert len(layer.free) + sum(len(o) for o in layer.owned) == layer.cache.k.shape[0]


def test_decode_module_runs(dev, capsys):
    decode.main()
    assert "step 200" in capsys.readouterr().out
