"""Scores that a call does not own, beside those that it adds to."""
import pytest
import torch

import int8_quantized_gb300 as q
from test_gpu_kv_cache import gen, make_cache, make_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("extra", [0, 2000])
@pytest.mark.parametrize("length,window,theirs", [(13, 0, [13, 14, 15]), (30, 11, [16, 17, 18]), (45, 5, [38, 39, 45, 46])])
def test_scores_outside_the_sequence_may_be_written_by_another_stream(dev, length, window, theirs, extra):
    """Tokens past the length and before the window, in the same 16 bytes as
    attended ones, take another stream's writes while the call runs."""
    g = gen(length)
    table, pages, _ = make_table(g, dev, [length], 16, extra=extra)
    c = make_cache(g, dev, pages, 2, 16, 64, "s8")
    qx = torch.randn((1, 8, 64), generator=g).to(dev)
    lengths = torch.tensor([length], dtype=torch.int32, device=dev)
    out = torch.empty_like(qx)
    ws = torch.empty(q.paged_attention_workspace_size(c, table, 8, True), dtype=torch.uint8, device=dev)
    page, off = table[0, torch.tensor(theirs, device=dev) // 16].long(), torch.tensor(theirs, device=dev) % 16
    marks = [torch.full((len(theirs), 2), float(i), device=dev) for i in range(300)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for mark in marks:
        q.paged_attention(c, table, lengths, qx, out, window=window, accumulate=True, workspace=ws, stream=side)
        c.score[page, :, off] = mark
    torch.cuda.synchronize()
    assert torch.equal(c.score[page, :, off], marks[-1])
    q.sync_status()
