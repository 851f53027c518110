"""The attention kernel's rings of tiles in shared memory: every form, with
tiles that are masked, cut and whole, gives the same bits each time.  A copy
that overtook a read of the slot it goes to would show as a change."""
import pytest
import torch

import int8_quantized_gb300 as q
from test_gpu_kv_cache import TYPES, gen, make_cache, make_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("page", [16, 24])
def test_attention_repeats_bit_for_bit(dev, page, G, D, qtype, cache):
    g = gen(D + G)
    lens = [3001, 17, 0, 1200, 640]
    table, pages, _ = make_table(g, dev, lens, page)
    c = make_cache(g, dev, pages, 2, page, D, cache)
    qx = torch.randn((len(lens), 2 * G, D), generator=g).to(TYPES[qtype]).to(dev)
    lengths = torch.tensor(lens, dtype=torch.int32, device=dev)
    ws = torch.empty(q.paged_attention_workspace_size(c, table, 2 * G, True), dtype=torch.uint8, device=dev)
    start = c.score.clone()
    first = None
    for _ in range(12):
        c.score.copy_(start)
        out, lse = torch.empty_like(qx), torch.empty(qx.shape[:2], device=dev)
        q.paged_attention(c, table, lengths, qx, out, lse=lse, window=1500, accumulate=True, workspace=ws)
        got = out.clone(), lse.clone(), c.score.clone()
        if first is None:
            first = got
        for a, b in zip(first, got):
            assert torch.equal(a, b)
    q.sync_status()
