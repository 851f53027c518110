"""The operators of a whole decode step together: 4-bit products around
kv_append with norms and paged attention, then logits and sampling; each part
against its plain form on what the part before it gave."""
import numpy as np
import pytest
import torch

import int8_quantized_gb300 as q
from int8_quantized_gb300 import decode
from test_gpu_kv_cache import host, reference_attention
from test_gpu_kv_norm import normed
from test_gpu_kv_cache import rotate
from test_gpu_nbits import dense, tolerance
from test_gpu_sample import kept_weights

pytestmark = pytest.mark.gpu


def matrix(g, rows, columns, dev, block=32):
    """A MatMulNBits and the same matrix in fp64: (codes less zero points), scales."""
    blocks = -(-rows // block)
    B = torch.randint(0, 256, (columns, blocks, block // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    s = ((torch.rand((columns, blocks), generator=g) + 0.5) / (4.6 * rows ** 0.5)).to(torch.bfloat16)
    z = torch.randint(0, 256, (columns, -(-blocks // 2)), generator=g, dtype=torch.int64).to(torch.uint8)
    w, sc = dense(B, s, z, rows, block)
    return q.MatMulNBits(B.to(dev), s.to(dev), rows, block, zero_points=z.to(dev)), w * sc


def check_product(x, y, w, K):
    x, y = x.cpu().double(), y.cpu().double()
    want = x @ w.t()
    assert ((y - want).abs() <= tolerance(x.abs() @ w.abs().t(), want, K, 32, "bf16", None)).all()


@pytest.mark.parametrize("B", [3, 12])  # by mma.sync, by tcgen05
def test_steps_with_4_bit_weights_norms_and_sampling(dev, B):
    g = torch.Generator()
    g.manual_seed(B)
    hidden, Hq, H, D, V = 256, 8, 2, 64, 5000
    qkv, w_qkv = matrix(g, hidden, (Hq + 2 * H) * D, dev)
    out, w_out = matrix(g, Hq * D, hidden, dev)
    lm, w_lm = matrix(g, hidden, V, dev)
    norms = [torch.randn((D,), generator=g) * 0.2 + 1 for _ in range(2)]
    turn = torch.arange(64, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2) / (D // 2))
    layer = decode.DecodeAttention(qkv, None, out, None, turn.cos().float().to(dev), turn.sin().float().to(dev), sequences=B,
                                   q_heads=Hq, kv_heads=H, head_dim=D, capacity=24, budget=12, sink=2, recent=4,
                                   q_norm=norms[0].to(dev), k_norm=norms[1].to(dev), norm_eps=1e-5)
    T, p = torch.full((B,), 0.7), torch.full((B,), 0.9)
    head = decode.TokenHead(lm, B, temperature=T.to(dev), top_p=p.to(dev))
    hid, kept = torch.empty((B, hidden), dtype=torch.bfloat16, device=dev), []
    before = {}
    plain = q.kv_append

    def watched(*args, **kw):  # (q is turned in place: what stood there before)
        before["qkv"] = layer.qkv.clone()
        return plain(*args, **kw)

    q.kv_append = watched
    try:
        for step in range(40):
            x = torch.randn((B, hidden), generator=g).to(torch.bfloat16).to(dev)
            layer.step(x, hid)
            check_product(x, before["qkv"], w_qkv, hidden)
            rows = before["qkv"].view(B, Hq + 2 * H, D).float().cpu()
            pos = np.full((1, B), step)
            cs = layer.cos.cpu().numpy(), layer.sin.cpu().numpy()
            want_q = rotate(normed(rows[:, :Hq], norms[0], 1e-5).numpy(), pos, *cs, None, False)
            got_q = layer.qkv.view(B, Hq + 2 * H, D)[:, :Hq]
            assert torch.equal(got_q.cpu(), torch.from_numpy(want_q).to(torch.bfloat16))
            key = rotate(normed(rows[:, Hq:Hq + H], norms[1], 1e-5).numpy(), pos, *cs, None, False)
            tab = layer.table.cpu().numpy()
            for b in range(B):
                t = layer.length[b] - 1
                pg, off = tab[b, t // layer.page], t % layer.page
                s = host(layer.cache.k_scale[pg, :, off])[:, None]
                assert np.all(np.abs(host(layer.cache.k[pg, :, off]) * s - key[b]) <= 0.501 * s)
            ref, *_ = reference_attention(layer.cache, layer.table, layer.length, got_q, 0, D ** -0.5)
            assert np.abs(host(layer.attended) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4
            check_product(layer.attended.view(B, -1), hid, w_out, Hq * D)
            u = torch.rand((B,), generator=g)
            tokens = head.step(hid, u.to(dev))
            check_product(hid, head.logits, w_lm, hidden)
            for b in range(B):
                w = kept_weights(head.logits[b].float().cpu().numpy(), float(T[b]), 0, float(p[b]))
                c = np.cumsum(w)
                assert int(tokens[b]) == int(np.searchsorted(c, np.float64(u[b]) * c[-1], side="right"))
            kept.append(tokens.tolist())
    finally:
        q.kv_append = plain
    q.sync_status()
    assert layer.position == [40] * B and max(max(layer.length), 12) <= 24
    assert len({tuple(t) for t in kept}) > 30


def test_a_matrix_of_the_wrong_size_is_refused(dev):
    g = torch.Generator()
    g.manual_seed(0)
    a, _ = matrix(g, 64, 256, dev)
    b, _ = matrix(g, 64, 128, dev)
    args = dict(sequences=1, q_heads=2, kv_heads=1, head_dim=64, capacity=20, budget=10, sink=1, recent=1)
    cos = torch.ones((8, 32), device=dev)
    with pytest.raises(ValueError, match="64 to 128 where 128 to 64"):
        decode.DecodeAttention(a, None, b, None, cos, cos, **args)
    with pytest.raises(ValueError, match="w_qkv must have 256"):
        decode.DecodeAttention(b, None, b, None, cos, cos, **args)
