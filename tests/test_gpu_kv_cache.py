"""The paged key/value cache on a GB300: kv_append, kv_gather,
paged_attention and kv_evict against plain numpy forms in 64 bits (and, where
every operation's rounding is fixed, bit for bit in 32).

Tolerances.  With u = 2^-24, a dot product of D terms has an error of at most
D u sum|q k| in any order, and twice that allows for the tensor pipe's
truncated sums; the score's factors (scale, softmax_scale, log2 e) add 4 u
|s|.  An error e in the scores changes a weight p by at most 2 e p, the
exponential adds 2^-21 p and a sum of L weights L u.  Weights rounded to 11
bits (bf16 queries, int8 cache) add 2^-11 p, to 16 bits 2^-16 p, and a bf16
output 2^-8 of itself.
"""
import math

import numpy as np
import pytest
import torch

import int8_quantized_gb300 as q

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def make_cache(g, dev, pages, heads, page, dim, cache, order="phtd", score=True):
    """Pools in memory order `order` (p page, h head, t token), as [p, h, t, d] views."""
    ext = {"p": pages, "h": heads, "t": page, "d": dim}
    perm = [order.index(a) for a in "phtd"]

    def pool(x):
        return x.permute(*[("phtd").index(a) for a in order]).contiguous().to(dev).permute(*perm)

    def per(x):
        o = order.replace("d", "")
        return x.permute(*["pht".index(a) for a in o]).contiguous().to(dev).permute(*[o.index(a) for a in "pht"])

    shape = [ext[a] for a in "phtd"]
    s = {}
    for n in ("k", "v"):
        x = torch.randn(shape, generator=g)
        if cache == "s8":
            s[n] = pool((x * 40).round().clamp(-128, 127).to(torch.int8))
            s[n + "_scale"] = per(torch.rand(shape[:3], generator=g) * 0.03 + 0.002)
        else:
            s[n] = pool(x.to(torch.bfloat16))
            s[n + "_scale"] = None
    s["score"] = per(torch.rand(shape[:3], generator=g)) if score else None
    return q.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["score"])


def make_table(g, dev, lens, page, spare=3, extra=0):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g)
    width = max(need + [1]) + extra
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return t.to(dev), sum(need) + spare, order[at:]


def host(x):
    return x.detach().cpu().to(torch.float64 if x.is_floating_point() else x.dtype).numpy()


def values(cache, name):
    x = host(getattr(cache, name)).astype(np.float64)
    s = getattr(cache, name + "_scale")
    return x if s is None else x * host(s)[..., None]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def reference_attention(cache, table, lens, qx, window, scale):
    k, v = values(cache, "k"), values(cache, "v")
    table, qx = table.cpu().numpy(), host(qx)
    page, H = k.shape[2], k.shape[1]
    B, Hq, D = qx.shape
    G = Hq // H
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    weight = np.zeros((B, Hq, D))           # sum p |v|
    err_s = np.zeros((B, Hq))
    probs = {}
    for b, n in enumerate(lens):
        t = np.arange(max(0, n - window) if window else 0, n)
        if not t.size:
            continue
        pg, off = table[b, t // page], t % page
        for h in range(Hq):
            kk, vv = k[pg, h // G, off], v[pg, h // G, off]
            s = kk @ qx[b, h] * scale
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            out[b, h], lse[b, h] = p @ vv, m + math.log(e.sum())
            weight[b, h] = p @ np.abs(vv)
            err_s[b, h] = 2 * D * U * (np.abs(kk) @ np.abs(qx[b, h])).max() * abs(scale) + 4 * U * np.abs(s).max()
            probs[b, h] = (pg, off, p)
    return out, lse, weight, err_s, probs


def check_attention(dev, lens, Hq, H, D, page, qtype, cache, window=0, accumulate=False, order="phtd", seed=0,
                    scale=None, strided=False, q_gain=2.0, change=None, extra=0):
    g = gen(seed)
    table, pages, _ = make_table(g, dev, lens, page, extra=extra)
    c = make_cache(g, dev, pages, H, page, D, cache, order)
    if change:
        change(c, table)
    B = len(lens)
    qx = (torch.randn((B, Hq, D), generator=g) * q_gain).to(TYPES[qtype]).to(dev)
    out = torch.full((B, Hq, D), 7.0, dtype=TYPES[qtype], device=dev)
    if strided:  # rows and heads inside wider tensors, at odd places
        wide = torch.zeros((B, Hq + 1, D + 3), dtype=TYPES[qtype], device=dev)
        wide[:, 1:, 3:] = qx
        qx = wide[:, 1:, 3:]
        out = torch.full((B, Hq + 1, D + 3), 7.0, dtype=TYPES[qtype], device=dev)[:, 1:, 3:]
    lse = torch.full((B, Hq), 7.0, device=dev)
    before = host(c.score)
    lengths = torch.tensor(lens, dtype=torch.int32, device=dev)
    s = D ** -0.5 if scale is None else scale
    q.paged_attention(c, table, lengths, qx, out, lse=lse, softmax_scale=scale, window=window, accumulate=accumulate)
    q.sync_status()
    ref, rlse, weight, err_s, probs = reference_attention(c, table, lens, qx, window, s)
    L = max(lens + [1])
    rel = 2 * err_s + 2.0 ** -21 + 2 * L * U
    narrow = 0.0 if qtype == "f32" else (2.0 ** -11 if cache == "s8" else 2.0 ** -16)
    tol = (rel + narrow)[..., None] * weight + (2.0 ** -8 if qtype == "bf16" else 2.0 ** -23) * np.abs(ref) + 1e-30
    got = host(out)
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))
    z = host(lse)
    empty = np.isinf(rlse)
    assert np.array_equal(np.isneginf(z), empty)
    ztol = err_s + 2.0 ** -21 + 2 * L * U + 2.0 ** -22 * np.abs(np.where(empty, 0, rlse))
    assert np.all(np.abs(z - rlse)[~empty] <= ztol[~empty])
    after = host(c.score)
    if not accumulate:
        assert np.array_equal(before, after)
        return
    want, stol = before.copy(), 2.0 ** -22 * np.abs(before) + 1e-30
    for (b, h), (pg, off, p) in probs.items():
        want[pg, h // (Hq // H), off] += p
        stol[pg, h // (Hq // H), off] += p * (rel[b, h] + err_s[b, h] + 2.0 ** -20)
    assert np.all(np.abs(after - want) <= stol), float(np.max(np.abs(after - want) / stol))


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 128, 144, 192, 256])
def test_attention_head_dims(dev, D, qtype, cache):
    check_attention(dev, [1, 37, 300], 8, 2, D, 16, qtype, cache, seed=D, accumulate=True)


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("page", [1, 5, 16, 24, 48, 128])
def test_attention_page_sizes(dev, page, cache):
    check_attention(dev, [130, 1, 67], 4, 2, 64, page, "bf16", cache, seed=page, accumulate=True)


@pytest.mark.parametrize("cache,qtype", [("s8", "bf16"), ("bf16", "bf16"), ("s8", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 9, 16, 17, 40])
def test_attention_shared_heads(dev, G, cache, qtype):
    check_attention(dev, [90, 33], G * 2, 2, 64, 16, qtype, cache, seed=G, accumulate=True)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257, 1000, 4097])
@pytest.mark.parametrize("accumulate", [False, True])
def test_attention_lengths(dev, n, accumulate):
    check_attention(dev, [n], 8, 2, 128, 16, "bf16", "s8", seed=n, accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
def test_attention_empty_sequences(dev, accumulate):
    check_attention(dev, [0, 0, 40, 0, 1, 0], 4, 4, 64, 16, "bf16", "s8", accumulate=accumulate)
    check_attention(dev, [0], 4, 4, 64, 16, "f32", "bf16", accumulate=accumulate)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 5000])
@pytest.mark.parametrize("cache", ["s8", "bf16"])
def test_attention_window(dev, window, cache):
    check_attention(dev, [1, 16, 99, 100, 101, 640, 0], 8, 2, 64, 24, "bf16", cache, window=window, accumulate=True,
                    seed=window)


@pytest.mark.parametrize("order", ["phtd", "pthd", "hptd", "tphd"])
@pytest.mark.parametrize("cache", ["s8", "bf16"])
def test_attention_orders_and_strides(dev, order, cache):
    check_attention(dev, [70, 200], 6, 3, 96, 16, "bf16", cache, order=order, accumulate=True, strided=True)
    check_attention(dev, [70, 200], 6, 3, 96, 20, "f32", cache, order=order, strided=True)


# Tables with room for long sequences: rows are then cut where the line says,
# not kept whole by a CTA.
CUT = [1, 0, 37, 300, 2000, 16, 700, 5]


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("qtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("G", [1, 5, 16])
def test_attention_cut_rows(dev, D, G, qtype, cache):
    check_attention(dev, CUT, 3 * G, 3, D, 16, qtype, cache, seed=D + G, accumulate=G != 5, extra=2000)


@pytest.mark.parametrize("cache,qtype", [("s8", "bf16"), ("bf16", "f32"), ("s8", "f32")])
@pytest.mark.parametrize("window", [0, 17, 250])
@pytest.mark.parametrize("page", [5, 24, 64])
def test_attention_cut_rows_pages_and_windows(dev, page, window, cache, qtype):
    check_attention(dev, CUT, 20, 1, 96, page, qtype, cache, window=window, seed=page, accumulate=True, extra=2000,
                    order="pthd", strided=True)


@pytest.mark.parametrize("lens", [[4000], [0, 0, 0], [1], [65] * 40, [5000, 1, 1, 1], [16 * 9] * 7])
def test_attention_cut_rows_lengths(dev, lens):
    check_attention(dev, lens, 8, 2, 128, 16, "bf16", "s8", accumulate=True, extra=2000)
    check_attention(dev, lens, 2, 2, 64, 16, "bf16", "bf16", extra=2000)


@pytest.mark.parametrize("G", [1, 4, 9, 32, 33, 40])
@pytest.mark.parametrize("page", [6, 16])
@pytest.mark.parametrize("B", [1, 30])
def test_attention_cut_rows_scores_in_one_launch_or_two(dev, G, page, B):
    """Tables that name up to 2^21 tokens of all heads, and more; up to 32 heads to one, and more."""
    for extra in (500, 140000):
        check_attention(dev, [900, 0, 77] * B, 2 * G, 2, 64, page, "bf16", "s8", accumulate=True, window=600,
                        extra=extra // B)


@pytest.mark.parametrize("G", [1, 9, 32, 33])
@pytest.mark.parametrize("page", [6, 16])
@pytest.mark.parametrize("extra", [4000, 140000])
def test_attention_cut_rows_scores_without_window(dev, G, page, extra):
    check_attention(dev, [900, 0, 77] * 3, 2 * G, 2, 64, page, "bf16", "s8", accumulate=True, extra=extra // 3)


@pytest.mark.parametrize("cache,qtype", [("s8", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("page", [7, 16])
@pytest.mark.parametrize("window", [1, 16, 17, 1000, 4500])
@pytest.mark.parametrize("G", [4, 20])
def test_attention_windows_of_long_sequences(dev, G, window, page, cache, qtype):
    """Windows within what a block takes whole, and above."""
    check_attention(dev, [5003, 0, 9000, 100, 16, 999], G, 1, 80, page, qtype, cache, window=window, seed=window,
                    accumulate=True, extra=1000)


@pytest.mark.parametrize("cache,qtype", [("s8", "bf16"), ("bf16", "bf16"), ("s8", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("D", [64, 112, 256])
@pytest.mark.parametrize("G", [1, 9, 20])
def test_attention_rows_shared_by_neighbouring_blocks(dev, G, D, cache, qtype):
    """Few rows of middling length, by two to eight blocks each."""
    for lens in ([640], [1500, 0, 37, 2900], [700] * 20):
        check_attention(dev, lens, G, 1, D, 16, qtype, cache, seed=G, accumulate=True)


def test_attention_cut_rows_over_many_sequences(dev):
    r = np.random.default_rng(5)
    check_attention(dev, [int(x) for x in r.integers(0, 200, 700)], 4, 2, 64, 16, "bf16", "s8", accumulate=True,
                    extra=300)
    check_attention(dev, [int(x) for x in r.integers(0, 20, 2500)], 2, 1, 16, 4, "f32", "bf16", extra=300)


@pytest.mark.parametrize("cache,qtype", [("s8", "bf16"), ("bf16", "f32")])
def test_attention_long(dev, cache, qtype):
    check_attention(dev, [40001, 3], 4, 1, 64, 32, qtype, cache, accumulate=True)


def test_attention_many_short_sequences(dev):
    r = np.random.default_rng(3)
    check_attention(dev, [int(x) for x in r.integers(0, 60, 300)], 4, 2, 64, 16, "bf16", "s8", accumulate=True)


def test_attention_more_sequences_than_one_schedule(dev):
    r = np.random.default_rng(4)
    check_attention(dev, [int(x) for x in r.integers(0, 4, 5000)], 1, 1, 16, 4, "bf16", "s8", accumulate=True)


@pytest.mark.parametrize("cache", ["s8", "bf16"])
def test_attention_sharp_scores(dev, cache):
    """Scores of hundreds: nearly all weight on one token, wherever it lies."""
    check_attention(dev, [500, 77], 8, 2, 128, 16, "f32", cache, q_gain=60.0, accumulate=True)
    check_attention(dev, [500, 77], 8, 2, 128, 16, "bf16", cache, q_gain=60.0, scale=-1.0)


def test_attention_rising_scores(dev):
    """Every tile raises the maximum, by little and by much."""
    for step in (0.01, 0.3, 5.0):
        def rise(c, table):
            n = table.shape[1] * c.k.shape[2]
            for t in range(n):
                pg = int(table[0, t // c.k.shape[2]])
                c.k[pg, :, t % c.k.shape[2]] = 0
                c.k[pg, :, t % c.k.shape[2], 0] = 100
                c.k_scale[pg, :, t % c.k.shape[2]] = step * t / 100
        check_attention(dev, [304], 2, 1, 64, 16, "bf16", "s8", change=rise, accumulate=True, scale=0.25)


@pytest.mark.parametrize("qtype", ["bf16", "f32"])
def test_attention_value_scales_far_apart(dev, qtype):
    """Value scales over many orders of magnitude, growing and shrinking along the sequence."""
    for sign in (1, -1):
        def spread(c, table):
            n = table.shape[1] * c.k.shape[2]
            for t in range(n):
                pg = int(table[0, t // c.k.shape[2]])
                c.v_scale[pg, :, t % c.k.shape[2]] = 10.0 ** (sign * (20.0 * t / n - 10.0))
        check_attention(dev, [160], 4, 2, 64, 16, qtype, "s8", change=spread)

    def zero(c, table):
        c.v_scale.zero_()
        c.k_scale[0].zero_()
    check_attention(dev, [160], 4, 2, 64, 16, qtype, "s8", change=zero, accumulate=True)


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_ignores_what_is_outside(dev, cache, bad):
    """Non-finite keys, values and scales before the window, past the end and
    in pages that no sequence names change nothing."""
    lens, window = [77, 5, 160], 40

    def spoil(c, table):
        page = c.k.shape[2]
        good = torch.zeros(c.k.shape[:3], dtype=torch.bool, device=dev)
        for b, n in enumerate(lens):
            for t in range(max(0, n - window), n):
                good[int(table[b, t // page]), :, t % page] = True
        if cache == "s8":
            c.k_scale[~good] = bad
            c.v_scale[~good] = bad
        else:
            c.k[~good] = bad
            c.v[~good] = bad
    check_attention(dev, lens, 8, 2, 64, 24, "bf16", cache, window=window, accumulate=True, change=spoil)


@pytest.mark.parametrize("cache", ["s8", "bf16"])
def test_attention_not_finite_inside(dev, cache):
    """A NaN key or value of an attended token reaches its own sequence and
    head, and nothing else."""
    g = gen(1)
    table, pages, _ = make_table(g, dev, [50, 50], 16)
    for name in ("k", "v"):
        c = make_cache(g, dev, pages, 2, 16, 64, cache)
        pg = int(table[0, 1])
        if cache == "s8":
            getattr(c, name + "_scale")[pg, 1, 3] = float("nan")
        else:
            getattr(c, name)[pg, 1, 3] = float("nan")
        qx = torch.randn((2, 4, 64), generator=g).to(dev)
        out = torch.empty_like(qx)
        q.paged_attention(c, table, torch.tensor([50, 50], dtype=torch.int32, device=dev), qx, out)
        bad = torch.isnan(out)
        assert bad[0, 2:].all() and not bad[0, :2].any() and not bad[1].any()


def test_attention_scores_of_minus_infinity(dev):
    """Tokens whose score is -infinity have no weight; others keep theirs."""
    g = gen(2)
    table, pages, _ = make_table(g, dev, [60], 16)
    c = make_cache(g, dev, pages, 1, 16, 64, "bf16")
    c.k[:] = c.k.abs()
    for t in list(range(0, 20)) + [33]:
        c.k[int(table[0, t // 16]), 0, t % 16] = float("-inf")
    qx = torch.rand((1, 2, 64), generator=g).to(dev) + 0.1
    out, lse = torch.empty_like(qx), torch.empty((1, 2), device=dev)
    q.paged_attention(c, table, torch.tensor([60], dtype=torch.int32, device=dev), qx, out, lse=lse, accumulate=True)
    t = np.array([t for t in range(20, 60) if t != 33])
    pg, off = table.cpu().numpy()[0, t // 16], t % 16
    k, v = host(c.k)[pg, 0, off], host(c.v)[pg, 0, off]
    for h in range(2):
        s = k @ host(qx)[0, h] / 8
        p = np.exp(s - s.max())
        assert np.allclose(host(out)[0, h], (p / p.sum()) @ v, rtol=0, atol=1e-4)
    assert torch.isfinite(c.score).all()


def test_attention_is_repeatable_and_stream_ordered(dev):
    g = gen(5)
    lens = [900, 30, 2500]
    table, pages, _ = make_table(g, dev, lens, 16)
    c = make_cache(g, dev, pages, 2, 16, 128, "s8")
    qx = torch.randn((3, 8, 128), generator=g).to(torch.bfloat16).to(dev)
    lengths = torch.tensor(lens, dtype=torch.int32, device=dev)
    ws = torch.empty(q.paged_attention_workspace_size(c, table, 8, True), dtype=torch.uint8, device=dev)
    start = c.score.clone()
    outs, scores = [], []
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, None, side):
        with torch.cuda.stream(side if stream is not None else torch.cuda.current_stream()):
            c.score.copy_(start)
            ws.fill_(0xEE)
            out = torch.empty_like(qx)
            q.paged_attention(c, table, lengths, qx, out, accumulate=True, workspace=ws, stream=stream)
            outs.append(out.clone())
            scores.append(c.score.clone())
        torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(scores[0], scores[1]) and torch.equal(scores[0], scores[2])


def test_attention_in_a_graph(dev):
    """Captured once, replayed with other lengths and queries."""
    g = gen(6)
    table, pages, _ = make_table(g, dev, [400, 400], 16)
    c = make_cache(g, dev, pages, 2, 16, 64, "s8")
    qx = torch.randn((2, 8, 64), generator=g).to(dev)
    lengths = torch.tensor([400, 400], dtype=torch.int32, device=dev)
    out = torch.empty_like(qx)
    ws = torch.empty(q.paged_attention_workspace_size(c, table, 8, False), dtype=torch.uint8, device=dev)
    q.paged_attention(c, table, lengths, qx, out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.paged_attention(c, table, lengths, qx, out, workspace=ws)
    for lens in ([3, 399], [0, 17], [256, 400]):
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        qx.copy_(torch.randn(qx.shape, generator=g))
        graph.replay()
        want = torch.empty_like(out)
        q.paged_attention(c, table, lengths, qx, want)
        assert torch.equal(out, want)


def test_attention_pool_past_32_bit_offsets(dev):
    """Pages whose elements lie past 2^32 in the pool."""
    D, page, H = 256, 128, 16
    pages = (1 << 32) // (D * page * H) + 40
    k = torch.zeros((pages, H, page, D), dtype=torch.int8, device=dev)
    v = torch.zeros_like(k)
    ks = torch.zeros((pages, H, page), device=dev)
    g = gen(8)
    last = torch.arange(pages - 8, pages)
    for t in (k, v):
        t[last] = torch.randint(-127, 128, (8, H, page, D), generator=g, dtype=torch.int8).to(dev)
    ks[last] = 0.01
    small = q.KVCache(k[last].clone(), v[last].clone(), ks[last].clone(), ks[last].clone(), ks[last].clone())
    big = q.KVCache(k, v, ks, ks.clone(), ks.clone())
    qx = torch.randn((2, H, D), generator=g).to(dev)
    lengths = torch.tensor([4 * page - 3, 4 * page], dtype=torch.int32, device=dev)
    outs = []
    for c, t in ((small, torch.arange(8).view(2, 4)), (big, last.view(2, 4))):
        out = torch.empty_like(qx)
        q.paged_attention(c, t.to(torch.int32).to(dev), lengths, qx, out, accumulate=True)
        outs.append(out)
    assert torch.equal(*outs) and torch.equal(small.score, big.score[last.to(dev)])
    # written and moved there too
    x = torch.randn((2, H, D), generator=g).to(dev)
    seq, index = torch.tensor([0, 1], dtype=torch.int32, device=dev), torch.tensor([5, 300], dtype=torch.int32, device=dev)
    for c, t in ((small, torch.arange(8).view(2, 4)), (big, last.view(2, 4))):
        t = t.to(torch.int32).to(dev)
        q.kv_append(c, t, seq, index, x, x)
        kept = torch.empty((1, H, 100), dtype=torch.int32, device=dev)
        q.kv_evict(c, t[:1], lengths[:1], t[1:], kept, sink=2, recent=5)
    assert torch.equal(small.k, big.k[last.to(dev)]) and torch.equal(small.v, big.v[last.to(dev)])


# ---------------------------------------------------------------------------
# append and gather
# ---------------------------------------------------------------------------
def rotate(x, positions, cos, sin, pair_axis, interleaved):
    """fp32, one rounding per operation (numpy)."""
    if cos is None:
        return x
    r = cos.shape[1]
    pos = positions[np.array(pair_axis), :].T if pair_axis is not None else np.repeat(positions[:1].T, r, 1)
    c, s = cos[pos, np.arange(r)][:, None], sin[pos, np.arange(r)][:, None]
    a, b = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def check_append(dev, T, Hq, H, D, page, type, cache, rot=0, axes=1, interleaved=False, order="phtd", seed=0,
                 strided=False, inplace=False, gain=1.0, edit=None, score=True, skip=()):
    g = gen(seed)
    lens = [T // 3 + 1, T, T // 2 + 2]
    table, pages, _ = make_table(g, dev, lens, page)
    c = make_cache(g, dev, pages, H, page, D, cache, order, score)
    seq = torch.randint(0, 3, (T,), generator=g)
    index = torch.zeros(T, dtype=torch.int64)
    seen = [0, 0, 0]
    for t in range(T):  # distinct places
        b = int(seq[t])
        while seen[b] >= lens[b]:
            b = (b + 1) % 3
        seq[t], index[t] = b, seen[b]
        seen[b] += 1
    dt = TYPES[type]
    qkv = (torch.randn((T, Hq + 2 * H, D), generator=g) * gain)
    if edit:
        edit(qkv)
    qkv = qkv.to(dt)
    if strided:
        wide = torch.zeros((T, Hq + 2 * H, D + 5), dtype=dt)
        wide[..., 5:] = qkv
        qkv_d = wide.to(dev)[..., 5:]
    else:
        qkv_d = qkv.to(dev)
    qx, kx, vx = qkv_d[:, :Hq], qkv_d[:, Hq:Hq + H], qkv_d[:, Hq + H:]
    kw, ref_rot = {}, (None,) * 4
    if rot:
        rows = 50
        ang = torch.rand((rows, rot // 2), generator=g, dtype=torch.float64) * 6.28
        cos, sin = ang.cos().float(), ang.sin().float()
        positions = torch.randint(0, rows, (axes, T), generator=g).to(torch.int32)
        pair_axis = [int(a) for a in torch.randint(0, axes, (rot // 2,), generator=g)] if axes > 1 else None
        kw = dict(positions=positions.to(dev), cos=cos.to(dev), sin=sin.to(dev), pair_axis=pair_axis,
                  interleaved=interleaved)
        ref_rot = (positions.numpy(), cos.numpy(), sin.numpy(), pair_axis)
    seq_d = seq.clone()
    for t in skip:
        seq_d[t] = -1
    before = {n: getattr(c, n).clone() for n in ("k", "v", "k_scale", "v_scale", "score") if getattr(c, n) is not None}
    q_in = qx.float().cpu().numpy()
    q_out = qx if inplace else torch.full((T, Hq, D), 9.0, dtype=dt, device=dev)
    old_q = q_out.clone()
    if Hq:
        kw.update(q=qx, q_out=q_out)
    q.kv_append(c, table, seq_d.to(torch.int32).to(dev), index.to(torch.int32).to(dev), kx, vx, **kw)
    q.sync_status()
    tab = table.cpu().numpy()
    live = [t for t in range(T) if t not in skip]
    pg, off = tab[seq.numpy(), index.numpy() // page], index.numpy() % page
    x = {"k": rotate(qkv[:, Hq:Hq + H].float().numpy(), *ref_rot, interleaved), "v": qkv[:, Hq + H:].float().numpy()}
    if Hq:
        want = torch.from_numpy(rotate(q_in, *ref_rot, interleaved)).to(dt)
        got = q_out.cpu()
        assert torch.equal(got[live], want[live])
        for t in skip:
            assert torch.equal(got[t], old_q.cpu()[t])
    for n in ("k", "v"):
        pool = before[n].cpu().clone()
        if cache == "bf16":
            pool[pg[live], :, off[live]] = bf16(x[n])[live]
            assert torch.equal(getattr(c, n).cpu(), pool)
            continue
        scale = np.abs(x[n]).max(-1) / np.float32(127)
        scale[scale == 0] = 1
        assert scale.dtype == np.float32
        code = np.clip(np.rint(x[n] / scale[..., None]), -128, 127).astype(np.int8)
        sp = before[n + "_scale"].cpu().clone()
        pool[pg[live], :, off[live]] = torch.from_numpy(code)[live]
        sp[pg[live], :, off[live]] = torch.from_numpy(scale)[live]
        assert torch.equal(getattr(c, n).cpu(), pool)
        assert torch.equal(getattr(c, n + "_scale").cpu(), sp)
        # and in 64 bits: half a step, a rounding of the quotient and one of the scale
        x64 = x[n].astype(np.float64)
        err = np.abs(code.astype(np.float64) * scale[..., None] - x64)
        assert np.all(err <= scale[..., None] * (0.5 + 128 * 2.0 ** -22))
    if score:
        sc = before["score"].cpu().clone()
        sc[pg[live], :, off[live]] = 0
        assert torch.equal(c.score.cpu(), sc)
    # read back
    for out_type in (torch.float32, torch.bfloat16):
        kb = torch.full((T, H, D), 3.0, dtype=out_type, device=dev)
        vb = torch.full((T, H, D + 1), 3.0, dtype=out_type, device=dev)[..., 1:]
        q.kv_gather(c, table, seq_d.to(torch.int32).to(dev), index.to(torch.int32).to(dev), kb, vb)
        q.sync_status()
        for n, back in (("k", kb), ("v", vb)):
            val = getattr(c, n).cpu().float()
            if cache == "s8":
                val = val * getattr(c, n + "_scale").cpu()[..., None]
            assert torch.equal(back.cpu()[live], val[pg[live], :, off[live]].to(out_type))
            for t in skip:
                assert (back[t] == 3.0).all()


@pytest.mark.parametrize("type", ["bf16", "f32"])
@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("D,rot", [(16, 16), (64, 32), (80, 80), (96, 30), (128, 128), (144, 2), (192, 64), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dev, D, rot, type, cache, interleaved):
    check_append(dev, 23, 4, 2, D, 16, type, cache, rot=rot, interleaved=interleaved, seed=D + rot)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("cache", ["s8", "bf16"])
def test_append_axes(dev, axes, cache):
    check_append(dev, 40, 6, 3, 128, 24, "bf16", cache, rot=96, axes=axes, seed=axes)


@pytest.mark.parametrize("T", [1, 2, 7, 300, 2500])
def test_append_tokens(dev, T):
    check_append(dev, T, 8, 2, 128, 16, "bf16", "s8", rot=128, seed=T)


@pytest.mark.parametrize("Hq,H", [(0, 1), (0, 5), (1, 1), (71, 1), (12, 12)])
def test_append_heads(dev, Hq, H):
    check_append(dev, 11, Hq, H, 64, 8, "bf16", "s8", rot=64 if Hq else 0)


@pytest.mark.parametrize("order", ["phtd", "pthd", "hptd", "tphd"])
def test_append_orders_strides_and_in_place(dev, order):
    check_append(dev, 50, 4, 2, 96, 5, "bf16", "s8", rot=96, order=order, strided=True)
    check_append(dev, 50, 4, 2, 96, 5, "f32", "bf16", rot=40, order=order, strided=True, inplace=True,
                 interleaved=True)
    check_append(dev, 50, 4, 2, 96, 5, "bf16", "s8", rot=96, order=order, inplace=True)


def test_append_padding_and_no_scores(dev):
    check_append(dev, 20, 4, 2, 64, 16, "bf16", "s8", rot=64, skip=(0, 7, 19), score=False)
    check_append(dev, 20, 4, 2, 64, 16, "f32", "bf16", skip=tuple(range(20)))


def test_append_extreme_rows(dev):
    """Zero rows, subnormal rows, one large element, ties and magnitudes from 1e-38 to 1e38."""
    def edit(x):
        x[0] = 0
        x[1] = 1e-42
        x[2] = 0
        x[2, :, 5] = -3.0
        x[3] = x[3] * 1e37
        x[4] = x[4] * 1e-37
        x[5] = torch.arange(x.shape[-1]).float() - 63.5       # ties
        x[5, :, 0] = 127.0
        x[6] = 1.0
    check_append(dev, 12, 2, 2, 128, 16, "f32", "s8", edit=edit)
    check_append(dev, 12, 2, 2, 128, 16, "bf16", "s8", edit=edit)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_append_not_finite(dev, bad):
    """A row with an infinity or a NaN gets a scale that is not finite; its neighbours are untouched."""
    g = gen(0)
    table, pages, _ = make_table(g, dev, [8], 16)
    c = make_cache(g, dev, pages, 2, 16, 64, "s8")
    x = torch.randn((8, 2, 64), generator=g)
    x[3, 1, 17] = bad
    x = x.to(dev)
    seq, index = torch.zeros(8, dtype=torch.int32, device=dev), torch.arange(8, dtype=torch.int32, device=dev)
    q.kv_append(c, table, seq, index, x, x)
    s = c.k_scale[int(table[0, 0]), :, :8].t()
    fine = torch.isfinite(s)
    assert not fine[3, 1] and fine.sum() == 15
    qx = torch.randn((1, 2, 64), generator=g).to(dev)
    out = torch.empty_like(qx)
    q.paged_attention(c, table, torch.tensor([8], dtype=torch.int32, device=dev), qx, out)
    assert torch.isfinite(out[0, 0]).all() and not torch.isfinite(out[0, 1]).any()


def test_append_no_tokens(dev):
    c = make_cache(gen(0), dev, 2, 2, 16, 64, "s8")
    e = torch.empty((0, 2, 64), device=dev)
    i = torch.empty(0, dtype=torch.int32, device=dev)
    t = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    q.kv_append(c, t, i, i, e, e)
    q.kv_gather(c, t, i, i, e, e.clone())
    q.sync_status()


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def reference_kept(score, n, budget, sink, recent):
    if n <= budget:
        return np.arange(n)
    x = np.where(np.isnan(score), -np.inf, score) + 0.0
    mid = np.arange(sink, n - recent)
    best = mid[np.lexsort((mid, -x[mid]))][:budget - sink - recent]
    return np.sort(np.concatenate((np.arange(sink), best, np.arange(n - recent, n))))


def check_evict(dev, lens, budget, sink, recent, H, D, page, cache, order="phtd", seed=0, change=None):
    g = gen(seed)
    keep = [min(n, budget) for n in lens]
    need = [-(-n // page) for n in keep]
    table, pages, free = make_table(g, dev, lens, page, spare=sum(need) + 2)
    width = -(-budget // page)
    new = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        new[b, :n] = free[at:at + n].to(torch.int32)
        at += n
    new = new.to(dev)
    c = make_cache(g, dev, pages, H, page, D, cache, order)
    if change:
        change(c, table)
    names = [n for n in ("k", "v", "k_scale", "v_scale", "score") if getattr(c, n) is not None]
    want = {n: getattr(c, n).cpu().clone() for n in names}
    kept = torch.full((len(lens), H, budget), 77, dtype=torch.int32, device=dev)
    new_lengths = torch.full((len(lens),), 77, dtype=torch.int32, device=dev)
    q.kv_evict(c, table, torch.tensor(lens, dtype=torch.int32, device=dev), new, kept, new_lengths, sink=sink,
               recent=recent)
    q.sync_status()
    assert new_lengths.tolist() == keep
    tab, new, got = table.cpu().numpy(), new.cpu().numpy(), kept.cpu().numpy()
    for b, n in enumerate(lens):
        t = np.arange(n)
        score = want["score"].numpy()[tab[b, t // page], :, t % page] if n else np.zeros((0, H))
        for h in range(H):
            r = reference_kept(score[:, h], n, budget, sink, recent)
            assert np.array_equal(got[b, h, :r.size], r) and (got[b, h, r.size:] == -1).all()
            j = np.arange(r.size)
            for x in names:
                src = want[x][tab[b, r // page], h, r % page].clone()
                want[x][new[b, j // page], h, j % page] = src
    for x in names:
        assert torch.equal(getattr(c, x).cpu().view(torch.int8 if x in "kv" and cache == "s8" else
                                                    torch.int16 if x in "kv" else torch.int32),
                           want[x].view(torch.int8 if x in "kv" and cache == "s8" else
                                        torch.int16 if x in "kv" else torch.int32))


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
def test_evict(dev, cache, D):
    check_evict(dev, [100, 33, 64, 0, 300], 48, 4, 10, 3, D, 16, cache, seed=D)


@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (17, 17, 0), (17, 0, 17), (17, 8, 9),
                                                (63, 1, 1), (64, 0, 0), (400, 4, 100)])
def test_evict_budgets(dev, budget, sink, recent):
    check_evict(dev, [64, 1, 65, 1000, 2], budget, sink, recent, 2, 32, 5, "s8", seed=budget)


@pytest.mark.parametrize("order", ["phtd", "pthd", "hptd", "tphd"])
def test_evict_orders(dev, order):
    check_evict(dev, [70, 200], 40, 2, 8, 3, 96, 24, "s8", order=order)
    check_evict(dev, [70, 200], 40, 2, 8, 3, 96, 24, "bf16", order=order)


@pytest.mark.parametrize("kind", ["equal", "two", "zeros", "special", "tiny", "negative"])
def test_evict_ties_and_special_scores(dev, kind):
    def change(c, table):
        s = c.score
        if kind == "equal":
            s.fill_(0.25)
        elif kind == "two":
            s.copy_((s > 0.5).float())
        elif kind == "zeros":
            s.copy_(torch.where(s > 0.5, 0.0, -0.0))
        elif kind == "special":
            u = s.clone()
            s[u < 0.2] = float("nan")
            s[(u >= 0.2) & (u < 0.4)] = float("-inf")
            s[u > 0.9] = float("inf")
        elif kind == "tiny":
            s.mul_(1e-42)
        else:
            s.copy_((s - 0.5) * 8).round_()
    check_evict(dev, [500, 90, 3000], 64, 3, 7, 2, 32, 16, "s8", change=change)


@pytest.mark.parametrize("n,budget", [(1024, 1023), (1025, 512), (20000, 3000), (70001, 65536)])
def test_evict_lengths(dev, n, budget):
    check_evict(dev, [n, n // 3], budget, 4, 33, 2, 16, 16, "s8", seed=n)


@pytest.mark.parametrize("rows", [1, 10, 20, 40])
@pytest.mark.parametrize("kind", ["drawn", "two"])
def test_evict_long_rows_by_one_to_eight_blocks(dev, rows, kind):
    # (of two values, so that many equal ones are taken in order across the blocks of a row)
    lens = [int(x) for x in np.random.default_rng(rows).integers(9000, 13500, rows)]
    lens[0] = 13501
    check_evict(dev, lens, 5000, 5, 100, 2, 16, 20, "s8", seed=rows,
                change=(lambda c, t: c.score.copy_((c.score > 0.7).float())) if kind == "two" else None)


@pytest.mark.parametrize("sink,recent", [(4, 33), (0, 0), (300, 700)])
def test_evict_more_keys_than_shared_memory_holds(dev, sink, recent):
    check_evict(dev, [400000], 1000, sink, recent, 1, 16, 256, "s8", seed=sink)


def test_evict_many(dev):
    r = np.random.default_rng(0)
    check_evict(dev, [int(x) for x in r.integers(0, 90, 400)], 24, 2, 5, 2, 16, 8, "bf16")


# ---------------------------------------------------------------------------
# indices out of range, found on the device
# ---------------------------------------------------------------------------
def reported(call):
    q.sync_status()
    call()
    with pytest.raises(q.I8QError) as e:
        q.sync_status()
    assert e.value.code == -1
    q.sync_status()


@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("page_id", [-1, 1 << 30])
def test_out_of_range_pages_are_left_out(dev, cache, page_id):
    """A page that the pools do not have counts as tokens that are not there."""
    g = gen(0)
    lens = [48, 48]
    table, pages, free = make_table(g, dev, lens, 16)
    c = make_cache(g, dev, pages, 2, 16, 64, cache)
    qx = torch.randn((2, 4, 64), generator=g).to(dev)
    lengths = torch.tensor(lens, dtype=torch.int32, device=dev)
    good = torch.empty_like(qx)
    short = table.clone()
    short[0, 1] = table[0, 2]
    q.paged_attention(c, short, torch.tensor([32, 48], dtype=torch.int32, device=dev), qx, good)
    bad = table.clone()
    bad[0, 1] = page_id
    out = torch.empty_like(qx)
    reported(lambda: q.paged_attention(c, bad, lengths, qx, out, accumulate=True))
    assert torch.equal(out[1], good[1]) and torch.allclose(out[0], good[0], rtol=0, atol=1e-4)
    x = torch.randn((3, 2, 64), generator=g).to(dev)
    seq = torch.tensor([0, 0, 1], dtype=torch.int32, device=dev)
    index = torch.tensor([20, 2, 1], dtype=torch.int32, device=dev)
    before = c.k.clone()
    reported(lambda: q.kv_append(c, bad, seq, index, x, x))
    changed = (c.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted({int(table[0, 0]), int(table[1, 0])})
    kb = torch.full_like(x, 5.0)
    reported(lambda: q.kv_gather(c, bad, seq, index, kb, kb.clone()))
    assert (kb[0] == 5.0).all() and (kb[1] != 5.0).any()
    kept = torch.empty((2, 2, 16), dtype=torch.int32, device=dev)
    new = free[:2].view(2, 1).to(torch.int32).to(dev)
    reported(lambda: q.kv_evict(c, bad, lengths, new, kept))
    before = c.k.clone()
    new[0, 0] = page_id
    reported(lambda: q.kv_evict(c, table, lengths, new, kept))
    changed = (c.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {int(new[1, 0])}


def test_evict_into_too_few_pages(dev):
    """A budget above what new_table names is fine while no sequence needs it;
    kept tokens without a place are left out."""
    g = gen(3)
    table, pages, free = make_table(g, dev, [20, 60], 16, spare=6)
    c = make_cache(g, dev, pages, 2, 16, 64, "s8")
    new = free[:4].view(2, 2).to(torch.int32).to(dev)
    lengths = torch.tensor([20, 30], dtype=torch.int32, device=dev)
    kept = torch.empty((2, 2, 1000), dtype=torch.int32, device=dev)
    q.kv_evict(c, table, lengths, new, kept)
    q.sync_status()
    assert (kept[0, :, :20] == torch.arange(20, device=dev)).all() and (kept[0, :, 20:] == -1).all()
    for t in (0, 15, 16, 29):
        assert torch.equal(c.k[new[1, t // 16], :, t % 16], c.k[table[1, t // 16], :, t % 16])
    before = c.k.clone()
    lengths[1] = 60
    reported(lambda: q.kv_evict(c, table, lengths, new, kept))
    changed = (c.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= set(new.flatten().tolist())
    for t in (0, 31):
        assert torch.equal(c.k[new[1, t // 16], :, t % 16], c.k[table[1, t // 16], :, t % 16])


def test_out_of_range_tokens_are_left_out(dev):
    g = gen(0)
    table, pages, _ = make_table(g, dev, [32, 32], 16)
    c = make_cache(g, dev, pages, 2, 16, 64, "s8")
    x = torch.randn((2, 2, 64), generator=g).to(dev)
    qo = torch.zeros_like(x)
    cos = torch.ones((8, 32), device=dev)
    ok = torch.tensor([0, 1], dtype=torch.int32, device=dev)
    for seq, index, pos in (([0, 2], [1, 1], [0, 0]), ([0, 1 << 30], [1, 1], [0, 0]), ([0, 1], [1, -1], [0, 0]),
                            ([0, 1], [1, 32], [0, 0]), ([0, 1], [1, 2 ** 31 - 1], [0, 0]), ([0, 1], [1, 1], [0, 8]),
                            ([0, 1], [1, 1], [0, -1])):
        t = [torch.tensor(v, dtype=torch.int32, device=dev) for v in (seq, index, pos)]
        before, qo = c.k.clone(), torch.zeros_like(x)
        c.k[int(table[0, 0]), :, 1] = 0
        reported(lambda: q.kv_append(c, table, t[0], t[1], x, x, q=x, q_out=qo, positions=t[2], cos=cos, sin=cos))
        assert (qo[0] != 0).any() and (qo[1] == 0).all()
        before[int(table[0, 0]), :, 1] = c.k[int(table[0, 0]), :, 1]
        assert torch.equal(before, c.k)
    q.kv_append(c, table, ok, ok, x, x)
    q.sync_status()


def test_out_of_range_lengths_are_cut(dev):
    g = gen(0)
    table, pages, _ = make_table(g, dev, [32, 32], 16)
    c = make_cache(g, dev, pages, 2, 16, 64, "s8")
    qx = torch.randn((2, 4, 64), generator=g).to(dev)
    out, want = torch.empty_like(qx), torch.empty_like(qx)
    q.paged_attention(c, table, torch.tensor([0, 32], dtype=torch.int32, device=dev), qx, want)
    reported(lambda: q.paged_attention(c, table, torch.tensor([-5, 2 ** 31 - 1], dtype=torch.int32, device=dev), qx, out))
    assert torch.equal(out, want)
