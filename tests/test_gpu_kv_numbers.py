"""How exactly attention holds its numbers: inputs on which a cut made on the
way shows, since ordinary ones hide it behind the outputs' own rounding.

Tolerances, with u = 2^-24.  Scores: a sum of D products in any order, rounded
or cut at each step, is off by at most 2 D u sum |q k|, and the factors
(scale, softmax_scale, log2 e) add 4 u |s|.  Weights: the exponential is good
to 2^-21, and sums of L weights to 2 L u, where nothing else is said."""
import math

import numpy as np
import pytest
import torch

import int8_quantized_gb300 as q
from test_gpu_kv_cache import TYPES, U, gen, host, make_cache, make_table, reference_attention

pytestmark = pytest.mark.gpu


def attend(dev, c, table, lens, qx, scale=None, accumulate=False, window=0):
    out, lse = torch.full_like(qx, 7.0), torch.full(qx.shape[:2], 7.0, device=dev)
    q.paged_attention(c, table, torch.tensor(lens, dtype=torch.int32, device=dev), qx, out, lse=lse,
                      softmax_scale=scale, accumulate=accumulate, window=window)
    q.sync_status()
    return out, lse


# ---- scores ----
@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_of_keys_with_one_large_channel(dev, D, G, qtype):
    """Channel 3 takes the whole range of the codes, and the others hold 0, 1
    and 2 (a row is scaled by its largest element); the query has one sign and
    elements of 2^-10 to 1.  The sum goes by D / 16 steps of the tensor pipe,
    each at most 4 u of it off (16 products and what was there, cut to one
    length), so D / 4 u where the general bound allows 2 D u."""
    g = gen(D + G)
    lens = [1, 7, 40, 300]
    table, pages, _ = make_table(g, dev, lens, 16, extra=1000 if G == 16 else 0)
    c = make_cache(g, dev, pages, 1, 16, D, "s8")
    c.k.copy_(torch.randint(0, 3, c.k.shape, generator=g, dtype=torch.int8))
    c.k[..., 3] = 127
    c.k_scale.fill_(0.25)
    qx = torch.exp2(-10 * torch.rand((4, G, D), generator=g)).to(TYPES[qtype]).to(dev)
    qx[..., 3] = 0
    before = host(c.score)
    out, lse = attend(dev, c, table, lens, qx, accumulate=True)
    _, want, _, err, probs = reference_attention(c, table, lens, qx, 0, D ** -0.5)
    err *= (D / 4 + 4) / (2 * D + 4)  # (no product is negative: sum |q k| is |s|)
    off = np.abs(host(lse) - want)
    tol = err + 2.0 ** -21 + 2 * np.array(lens)[:, None] * U + 2.0 ** -22 * np.abs(want)
    assert np.all(off <= tol), float((off / tol).max())
    score, stol = before.copy(), 2.0 ** -22 * np.abs(before)
    for (b, h), (pg, at, p) in probs.items():
        score[pg, 0, at] += p
        stol[pg, 0, at] += p * (3 * err[b, h] + 2.0 ** -20 + 2 * lens[b] * U)
    off = np.abs(host(c.score) - score)
    assert np.all(off <= stol), float((off / np.maximum(stol, 1e-30)).max())


@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("cache,log2", [("s8", -100), ("s8", -40), ("s8", 60), ("s8", 100), ("s8", 110), ("bf16", -100),
                                        ("bf16", -40), ("bf16", 60), ("bf16", 100)])
def test_scores_of_very_large_and_small_queries(dev, log2, qtype, cache):
    """Powers of two taken from the keys and given to the query change nothing
    (while all products with the keys' scales, and the keys, are normal numbers)."""
    g = gen(7)
    table, pages, _ = make_table(g, dev, [50], 16)
    c = make_cache(g, dev, pages, 1, 16, 64, cache)
    qx = torch.randn((1, 4, 64), generator=g).to(TYPES[qtype]).to(dev)
    want, wlse = attend(dev, c, table, [50], qx)
    if cache == "s8":
        c.k_scale.mul_(2.0 ** -log2)
    else:
        c.k.mul_(2.0 ** -log2)
    out, lse = attend(dev, c, table, [50], qx * 2.0 ** log2)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("ratio", [10, 16, 20, 24])
def test_scores_of_queries_with_one_large_element(dev, ratio, qtype):
    """One element of the query is 2^ratio times the others, where the keys are 0."""
    g = gen(ratio)
    lens = [1, 30]
    table, pages, _ = make_table(g, dev, lens, 16)
    c = make_cache(g, dev, pages, 1, 16, 64, "s8")
    c.k[..., 5] = 0
    qx = torch.randn((2, 4, 64), generator=g).to(TYPES[qtype]).to(dev)
    qx[..., 5] = 2.0 ** ratio
    out, lse = attend(dev, c, table, lens, qx)
    _, want, _, err, _ = reference_attention(c, table, lens, qx, 0, 0.125)
    off = np.abs(host(lse) - want)
    tol = err + 2.0 ** -21 + 2 * np.array(lens)[:, None] * U + 2.0 ** -22 * np.abs(want)
    assert np.all(off <= tol), float((off / tol).max())


# ---- weights ----
@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weighted_values_that_cancel(dev, D, G, qtype):
    """Equal scores, and three tokens whose values add up to nothing: a c + b c
    - (a + b) c.  What is left is what the products with a, b and a + b lost,
    at most 2^-24 of each, and the sums' 3 u."""
    B = 64
    g = gen(D)
    table, pages, _ = make_table(g, dev, [3] * B, 16)
    c = make_cache(g, dev, pages, 1, 16, D, "s8")
    c.k.zero_()
    tab = table[:, 0].long()
    code = torch.randint(1, 128, (B, D), generator=g, dtype=torch.int8).to(dev)
    for t, sign in enumerate((1, 1, -1)):
        c.v[tab, 0, t] = code * sign
    a = (torch.randint(1 << 22, 1 << 23, (2, B), generator=g).double() * 2.0 ** -24).to(dev)  # 23 bits: a + b is exact
    c.v_scale[tab, 0, 0], c.v_scale[tab, 0, 1], c.v_scale[tab, 0, 2] = a[0].float(), a[1].float(), (a[0] + a[1]).float()
    qx = torch.randn((B, G, D), generator=g).to(TYPES[qtype]).to(dev)
    out, _ = attend(dev, c, table, [3] * B, qx)
    weight = (2 / 3 * (a[0] + a[1])[:, None] * code.double()).cpu().numpy()[:, None]
    off = np.abs(host(out))
    tol = (2.0 ** -24 + 3 * U) * weight + 1e-30
    assert np.all(off <= tol), float((off / tol).max())


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("G", [4, 16])
def test_sums_of_long_rows_are_rounded(dev, G, cache):
    """256 sequences of 131072 tokens (the same few pages over and over) of two
    scores, so that weights have all their bits, and values of one sign but
    for one token's, which takes their sum away.  Sums that are rounded are off
    by u sqrt(n) or so (n <= 8192 tiles), with 8 for the tails; sums that are
    cut lose u / 2 and more at every step, always downwards."""
    g = gen(3)
    L, D, page, B = 131072, 64, 128, 256
    pages = 9
    c = make_cache(g, dev, pages, 1, page, D, cache, score=False)
    table = torch.randint(0, 8, (B, L // page), generator=g, dtype=torch.int32)
    table[:, 0] = 8
    c.k.zero_()
    c.k[:, 0, 0, 0] = 1
    w = torch.ones((pages, page), dtype=torch.float64)
    w[:, 0] = math.exp(5.59375 / 8)
    if cache == "s8":
        c.k_scale.fill_(1.0)
        c.v.fill_(93)
        c.v_scale.copy_(0.5 + torch.rand(c.v_scale.shape, generator=g) / 2)
        one = c.v_scale.double().cpu()[:, 0] * 93
    else:
        c.v.copy_((0.5 + torch.rand(c.v.shape[:3], generator=g) / 2)[..., None].to(torch.bfloat16))
        one = c.v[:, 0, :, 0].double().cpu()
    # the first token of each sequence (page 8) takes their mean sum away, the rest is the reference's
    away = float((one * w).sum(-1)[:8].mean() * (L // page) / w[8, 0])
    if cache == "s8":
        c.v[8, 0, 0] = -127
        c.v_scale[8, 0, 0] = away / 127
        one[8, 0] = -127 * c.v_scale[8, 0, 0].double().cpu()
    else:
        c.v[8, 0, 0] = -away
        one[8, 0] = c.v[8, 0, 0, 0].double().cpu()
    total = w.sum(-1)[table.long()].sum(-1)
    want = (one * w).sum(-1)[table.long()].sum(-1) / total
    weight = (one.abs() * w).sum(-1)[table.long()].sum(-1) / total
    qx = torch.randn((B, G, D), generator=g)
    qx[..., 0] = 5.59375
    qx = qx.to(torch.bfloat16).to(dev)
    out, _ = attend(dev, c, table.to(dev), [L] * B, qx)
    off = (out.double().cpu() - want[:, None, None]).abs()
    tol = (8 * math.sqrt(8192) * U * weight + 2.0 ** -8 * want.abs())[:, None, None]
    assert bool((off <= tol).all()), float((off / tol).max())


# ---- what is not finite ----
@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [64, 80])
def test_an_infinite_key_is_not_passed_over(dev, D, bad, sign, qtype):
    """A key with an infinite element, written by kv_append beside finite
    values: its scale is infinite, and what attends to it is not finite,
    whatever the sign of the query there."""
    g = gen(0)
    table, pages, _ = make_table(g, dev, [8, 8], 16)
    c = make_cache(g, dev, pages, 2, 16, D, "s8")
    k, v = torch.randn((16, 2, D), generator=g), torch.randn((16, 2, D), generator=g)
    k[3, 1, 17] = bad
    seq = torch.arange(16, device=dev, dtype=torch.int32) // 8
    index = torch.arange(16, device=dev, dtype=torch.int32) % 8
    c.score.fill_(1.0)
    q.kv_append(c, table, seq, index, k.to(dev), v.to(dev))
    qx = torch.randn((2, 4, D), generator=g).to(TYPES[qtype]).to(dev)
    qx[..., 17] = sign
    out, lse = attend(dev, c, table, [8, 8], qx, accumulate=True)
    good = torch.ones((2, 4), dtype=torch.bool, device=dev)
    good[0, 2:] = False
    assert torch.equal(torch.isfinite(lse), good)
    assert torch.equal(torch.isfinite(out), good[..., None].expand_as(out))
    score = c.score[table[:, 0].long(), :, :8]
    assert torch.isfinite(score[1]).all() and torch.isfinite(score[0, 0]).all() and not torch.isfinite(score[0, 1]).any()
