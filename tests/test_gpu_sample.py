"""sample on a GB300 against the definition in 64 bits, token by token.

Weights here are fp64's exponentials (2^-52) and the library's are off by
2^-42; both are compared at random numbers in the middle of each kept token's
interval, as fp32 holds it, and where that is not as wide as 2^-22 the token is
left out.  A kept set's border is met by a top_p or min_p that is 1e-9 from no
prefix's share.  Log-probabilities: the logarithm of a ratio rounded thrice
(3 2^-24) and of its own rounding, 2 units in its last place."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import int8_quantized_gb300 as q

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def kept_weights(x, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """fp64 weights of a row's kept tokens by index, 0 for the others."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    top = x.max()
    with np.errstate(invalid="ignore"):
        w = np.exp((x - top) / np.float64(T))
    w[x == top] = 1.0
    w[np.isneginf(x)] = 0.0
    if np.isposinf(top):
        w[x != top] = 0.0
    order = np.lexsort((np.arange(x.size), -x))
    n = x.size
    if 0 < top_k < n:
        n = top_k
    ws = w[order]
    if top_p < 1.0:
        c = np.cumsum(ws[:n])
        n = min(n, int(np.searchsorted(c, np.float64(np.float32(top_p)) * c[-1], side="left")) + 1)
    n = min(n, int((ws >= np.float64(np.float32(min_p))).sum()))
    n = max(n, 1)
    out = np.zeros_like(w)
    out[order[:n]] = ws[:n]
    return out


def rows_of(x, R, dtype, dev):
    return torch.from_numpy(np.tile(x, (R, 1))).to(dtype).to(dev)


def per_row(v, R, dtype, dev):
    return None if v is None else torch.full((R,), v, dtype=dtype, device=dev)


def call(dev, logits, u, T=None, top_k=None, top_p=None, min_p=None, **kw):
    R = logits.shape[0]
    tokens = torch.full((R,), -7, dtype=torch.int32, device=dev)
    logp = torch.full((R,), 7.0, device=dev)
    q.sample(logits, u, tokens, logprobs=logp, temperature=per_row(T, R, torch.float32, dev),
             top_k=per_row(top_k, R, torch.int32, dev), top_p=per_row(top_p, R, torch.float32, dev),
             min_p=per_row(min_p, R, torch.float32, dev), **kw)
    return tokens, logp


def check(dev, x, type="f32", T=1.0, top_k=None, top_p=None, min_p=None, most=300, seed=0):
    """Every kept token (`most` of them) by the middle of its interval."""
    x = torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[type]).float().numpy()
    T = float(np.float32(T))
    w = kept_weights(x, T, top_k or 0, 1.0 if top_p is None else top_p, min_p or 0.0)
    c = np.cumsum(w)
    lo, hi = (c - w) / c[-1], c / c[-1]
    mid = ((lo + hi) / 2).astype(np.float32)
    ids = np.nonzero((w > 0) & (hi - lo > 2.0 ** -22) & (mid < 1))[0]
    if ids.size > most:
        ids = np.random.default_rng(seed).choice(ids, most, replace=False)
    assert ids.size
    logits = rows_of(x, ids.size, TYPES[type], dev)
    tokens, logp = call(dev, logits, torch.from_numpy(mid[ids]).to(dev), T, top_k, top_p, min_p)
    q.sync_status()
    assert np.array_equal(tokens.cpu().numpy(), ids)
    want = np.log(w[ids] / c[-1])
    tol = 4 * 2.0 ** -24 + 2.0 ** -23 * np.abs(want)
    assert np.all(np.abs(logp.cpu().double().numpy() - want) <= tol)


def logits_of(V, spread=2.0, seed=0):
    return np.random.default_rng(seed).normal(0, spread, V).astype(np.float32)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 100, 1000, 4097, 8192, 33001, 131072, 200000])
def test_vocabularies(dev, V, type):
    x = logits_of(V, seed=V)
    check(dev, x, type, most=4)       # few rows: a cluster each
    check(dev, x, type, T=0.7, top_p=0.9, most=4)
    check(dev, x, type, T=0.5, top_k=min(V, 40), top_p=0.8, min_p=0.01, most=200)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("top_k", [1, 2, 10, 500, 2999, 3000, 3001, 0, -1])
def test_top_k(dev, type, top_k):
    check(dev, logits_of(3000, seed=1), type, top_k=top_k)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("top_p", [0.0, 1e-30, 0.01, 0.3, 0.77, 0.95, 0.9999, 1.0, 1.5])
@pytest.mark.parametrize("top_k", [None, 3, 100])
def test_top_p(dev, type, top_p, top_k):
    check(dev, logits_of(2500, seed=2), type, T=0.9, top_p=top_p, top_k=top_k)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("min_p", [0.0, 1e-20, 0.001, 0.05, 0.5, 0.999, 1.0])
def test_min_p(dev, type, min_p):
    check(dev, logits_of(2500, seed=3), type, T=1.1, min_p=min_p)
    check(dev, logits_of(2500, seed=4), type, T=1.1, min_p=min_p, top_p=0.97, top_k=900)


@pytest.mark.parametrize("T", [1e-3, 0.05, 0.3, 1.0, 3.0, 50.0, 1e30, float("inf"), 1e-40])
def test_temperatures(dev, T):
    check(dev, logits_of(1500, seed=5), "f32", T=T)
    check(dev, logits_of(1500, seed=5), "bf16", T=T, top_p=0.9)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_equal_logits(dev, type):
    """Borders inside a run of equal logits: the lowest indices are kept."""
    x = np.zeros(5000, np.float32)
    check(dev, x, type, most=200)
    check(dev, x, type, top_k=77)
    check(dev, x, type, top_p=0.1)      # fp32(0.1) is above a tenth: 501 tokens
    x[::3] = 1.0
    check(dev, x, type, top_k=1700)     # 1667 of the larger, 33 of the others
    check(dev, x, type, top_p=0.75, T=0.5)
    check(dev, x, type, top_k=2000, top_p=0.99)
    x = np.repeat(np.array([3.0, -1.0, 2.0, 3.0], np.float32), 700)
    for k in (1, 699, 700, 701, 1400, 1401, 2100, 2101):
        check(dev, x, type, top_k=k, most=100)


def test_the_random_number_at_a_border(dev):
    """Equal weights: the running sum has to exceed random times the whole."""
    x = torch.zeros((9, 8), device=dev)
    u = torch.tensor([0.0, 0.124, 0.125, 0.126, 0.25, 0.5, 0.875, 0.999, 1 - 2.0 ** -24], device=dev)
    tokens, logp = call(dev, x, u)
    assert tokens.tolist() == [0, 0, 1, 1, 2, 4, 7, 7, 7]
    assert (logp == math.log(1 / 8)).all()
    x[:, 2:] = -math.inf
    assert call(dev, x, u)[0].tolist() == [0, 0, 0, 0, 0, 1, 1, 1, 1]


def test_special_logits(dev):
    inf, low = math.inf, torch.finfo(torch.float32).min
    x = torch.randn((8, 300), device=dev)
    x[0] = -inf
    x[1] = math.nan
    x[2, :] = -inf
    x[2, 299] = -5.0
    x[3, 17] = x[3, 200] = inf
    x[4, 100] = math.nan
    x[5] = low
    x[5, 3] = 0.0
    x[6] = low                      # (the type's lowest value everywhere: a number like any other)
    x[7] = torch.finfo(torch.float32).max
    x[7, :150] = low
    u = torch.tensor([0.3, 0.3, 0.3, 0.6, 0.5, 0.999, 0.5, 0.0], device=dev)
    for kw in ({}, dict(top_p=0.9), dict(top_k=200), dict(top_k=5, top_p=0.5, min_p=0.1, T=0.5)):
        tokens, logp = call(dev, x, u, **kw)
        q.sync_status()
        t, lp = tokens.tolist(), logp.tolist()
        assert t[:3] == [-1, -1, 299] and lp[:2] == [-inf, -inf] and lp[2] == 0.0
        assert t[3] == (200 if kw.get("top_p") != 0.5 else 17)
        assert t[5] == 3 and lp[5] == 0.0
        assert t[7] == 150
        assert t[4] != 100
        if not kw:
            assert t[6] == 150 and abs(lp[6] + math.log(300)) < 1e-6


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_greedy_and_mixed_rows(dev, type):
    R, V = 70, 5003
    g = torch.Generator()
    g.manual_seed(1)
    x = (torch.randn((R, V), generator=g) * 3).to(TYPES[type])
    x[5, 100] = x[5, 4000] = 50.0
    T = torch.rand((R,), generator=g) + 0.3
    T[::5] = 0.0
    k = torch.randint(0, 3000, (R,), generator=g).to(torch.int32)
    p, m = torch.rand((R,), generator=g) * 1.2, torch.rand((R,), generator=g) * 0.1
    u = torch.rand((R,), generator=g)
    tokens = torch.empty((R,), dtype=torch.int32, device=dev)
    logp = torch.empty((R,), device=dev)
    q.sample(x.to(dev), u.to(dev), tokens, logp, T.to(dev), k.to(dev), p.to(dev), m.to(dev))
    q.sync_status()
    for r in range(R):
        row = x[r].float().numpy()
        if T[r] == 0:
            assert tokens[r] == int(np.argmax(row)) and logp[r] == 0
            continue
        w = kept_weights(row, float(T[r]), int(k[r]), float(p[r]), float(m[r]))
        c = np.cumsum(w)
        t = int(np.searchsorted(c, np.float64(u[r]) * c[-1], side="right"))
        assert tokens[r] == t
        assert abs(float(logp[r]) - math.log(w[t] / c[-1])) <= 2e-6
    only = torch.empty_like(tokens)  # the smallest call
    q.sample(x.to(dev), u.to(dev), only)
    w = [kept_weights(x[r].float().numpy()) for r in range(R)]
    assert only.tolist() == [int(np.searchsorted(np.cumsum(a), np.float64(u[r]) * np.cumsum(a)[-1], side="right"))
                             for r, a in enumerate(w)]


@pytest.mark.parametrize("rows", [1, 3, 19, 40, 80, 160, 400])
def test_clusters_of_every_size(dev, rows):
    V = 40001
    x = torch.from_numpy(logits_of(rows * V, 1.0, rows).reshape(rows, V))
    u = torch.from_numpy(np.random.default_rng(rows).random(rows).astype(np.float32))
    for type in ("f32", "bf16"):
        y = x.to(TYPES[type])
        tokens, _ = call(dev, y.to(dev), u.to(dev), T=0.8, top_p=0.9)
        q.sync_status()
        for r in range(0, rows, max(1, rows // 8)):
            w = kept_weights(y[r].float().numpy(), float(np.float32(0.8)), 0, 0.9)
            c = np.cumsum(w)
            assert int(tokens[r]) == int(np.searchsorted(c, np.float64(u[r]) * c[-1], side="right"))


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (3, 4), (5, 1), (7, 9)])
def test_strides_and_alignment(dev, type, offset, pad):
    V = 1003
    x = torch.from_numpy(logits_of(6 * V, 3.0, 7).reshape(6, V)).to(TYPES[type])
    wide = torch.full((6, offset + V + pad), 100.0, dtype=x.dtype, device=dev)
    rows = wide[:, offset:offset + V]
    rows.copy_(x)
    u = torch.tensor([0.0, 0.2, 0.5, 0.7, 0.9, 0.99], device=dev)
    a, la = call(dev, rows, u, T=0.9, top_k=300, top_p=0.99)
    b, lb = call(dev, x.to(dev), u, T=0.9, top_k=300, top_p=0.99)
    q.sync_status()
    assert torch.equal(a, b) and torch.equal(la, lb)
    w = kept_weights(x[2].float().numpy(), float(np.float32(0.9)), 300, 0.99)
    assert int(a[2]) == int(np.searchsorted(np.cumsum(w), 0.5 * np.cumsum(w)[-1], side="right"))


def test_weights_of_a_large_flat_vocabulary(dev):
    """2^20 tokens: sums of 62 bits."""
    V = 1 << 20
    x = np.zeros(V, np.float32)
    check(dev, x, "bf16", most=3)
    x = logits_of(V, 0.01, 3)
    check(dev, x, "f32", most=3, top_p=0.5)


def test_out_of_range_settings_are_reported(dev):
    x = torch.randn((1, 50), device=dev)
    good = dict(T=1.0, top_p=0.9, min_p=0.1)
    for u, bad in ((0.5, dict(T=-1.0)), (0.5, dict(T=math.nan)), (0.5, dict(top_p=-0.1)), (0.5, dict(top_p=math.nan)),
                   (0.5, dict(min_p=-0.1)), (0.5, dict(min_p=1.1)), (0.5, dict(min_p=math.nan)), (1.0, {}), (-0.1, {}),
                   (math.nan, {})):
        kw = dict(good)
        kw.update(bad)
        tokens, logp = call(dev, x, torch.tensor([u], device=dev), **kw)
        with pytest.raises(q.I8QError, match="sample met") as e:
            q.sync_status()
        assert e.value.code == -1
        assert tokens.item() == -1 and math.isnan(logp.item())
    two = torch.randn((2, 50), device=dev)
    tokens, logp = call(dev, two, torch.tensor([1.0, 0.5], device=dev))
    with pytest.raises(q.I8QError):
        q.sync_status()
    assert tokens[0] == -1 and tokens[1] >= 0 and logp[1] < 0  # its neighbour is drawn
    q.sync_status()


def test_streams_and_graphs(dev):
    R, V = 20, 32001
    x = torch.randn((R, V), device=dev) * 3
    u = torch.rand((R,), device=dev)
    one, lp = call(dev, x, u, T=0.8, top_p=0.95)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two, _ = call(dev, x, u, T=0.8, top_p=0.95)
    T, p = torch.full((R,), 0.8, device=dev), torch.full((R,), 0.95, device=dev)
    three = torch.zeros_like(one)
    side.wait_stream(torch.cuda.current_stream())
    q.sample(x, u, three, temperature=T, top_p=p, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(one, three)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.sample(x, u, three, temperature=T, top_p=p)
    other = torch.randn((R, V), device=dev)
    x.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(three, call(dev, other, u, T=0.8, top_p=0.95)[0])


def test_no_rows_and_refusals(dev):
    x, u = torch.randn((3, 50), device=dev), torch.rand((3,), device=dev)
    t = torch.full((3,), 5, dtype=torch.int32, device=dev)
    q.sample(x[:0], u[:0], t[:0])
    for args, err, match in (((x[0], u, t), ValueError, "logits must be"), ((x.half(), u, t), TypeError, "float32"),
                             ((x.cpu(), u, t), TypeError, "CUDA"), ((x, u[:2], t), ValueError, "random must have"),
                             ((x, u.double(), t), TypeError, "random must be"), ((x, u, t.long()), TypeError, "tokens must be"),
                             ((x.t().contiguous().t(), u, t), ValueError, "contiguous rows"),
                             ((x[:1].expand(3, 50), u, t), q.I8QError, "overlap")):
        with pytest.raises(err, match=match):
            q.sample(*args)
    for kw in (dict(temperature=u.double()), dict(top_k=u), dict(top_p=0.9), dict(min_p=u.cpu()), dict(logprobs=t)):
        with pytest.raises(TypeError, match="must be a contiguous"):
            q.sample(x, u, t, **kw)
    torch.cuda.synchronize()
    assert (t == 5).all()


@pytest.mark.parametrize("kw", [{}, dict(T=0.7, top_p=0.8), dict(T=0.5, top_k=3000, top_p=0.9, min_p=0.001), dict(top_k=33000 - 5)])
def test_many_long_rows_of_odd_values(dev, kw):
    """Rows whose weights come from a table, and what the table does not hold:
    zeros, numbers below 2^-16 and from 2^7 on, infinities, NaN, masks, and runs
    of equal logits longer than a list."""
    R, V = 160, 33000
    x = torch.from_numpy(logits_of(R * V, 2.0, 9).reshape(R, V))
    g = torch.Generator()
    g.manual_seed(2)
    some = torch.rand((R, V), generator=g)
    x[0:20][some[0:20] < 0.5] = 0.0
    x[20:40] *= 1e-6
    x[40:60] *= 100.0
    x[60:80][some[60:80] < 0.9] = -math.inf
    x[80:100][some[80:100] < 0.3] = math.nan
    x[100:120] = 2.0
    x[120:130, 5::7] = math.inf
    x[130:140] = x[130:140].round()
    x[140:150][some[140:150] < 0.5] = torch.finfo(torch.bfloat16).min
    x[150] = -math.inf
    x = x.to(torch.bfloat16)
    u = torch.rand((R,), generator=g)
    tokens, logp = call(dev, x.to(dev), u.to(dev), **kw)
    q.sync_status()
    T = float(np.float32(kw.get("T", 1.0)))
    for r in range(0, 151, 3):
        if r == 150:
            assert int(tokens[r]) == -1
            continue
        w = kept_weights(x[r].float().numpy(), T, kw.get("top_k", 0), kw.get("top_p", 1.0), kw.get("min_p", 0.0))
        c = np.cumsum(w)
        assert int(tokens[r]) == int(np.searchsorted(c, np.float64(u[r]) * c[-1], side="right")), r


@pytest.mark.parametrize("T", [1e-5, 3e-4, 1e-2])
@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_sharp_temperatures_of_large_logits(dev, type, T):
    """Logits so near each other, and so far from 0, that a step of the histogram is below one of theirs."""
    rng = np.random.default_rng(3)
    x = (100.0 + rng.integers(-40, 40, 9000) * 2.0 ** -17).astype(np.float32)
    check(dev, x, type, T=T, top_p=0.9, most=100)
    check(dev, x, type, T=T, top_k=500, top_p=0.7, most=100)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("V", [8192, 8193, 16384, 20000, 32768, 33000])
def test_the_shortest_shares_of_a_cluster(dev, V, type):
    """2, 4 and 8 CTAs with 4096 tokens or few more each, call behind call: a
    CTA may not hand its largest logit to one that has not started."""
    R = 5
    x = torch.from_numpy(logits_of(R * V, 2.0, V).reshape(R, V)).to(TYPES[type])
    u = torch.from_numpy(np.random.default_rng(V).random(R).astype(np.float32))
    T = torch.full((R,), 0.9)
    T[3] = 0.0
    want = []
    for r in range(R):
        w = kept_weights(x[r].float().numpy(), float(T[r]) or 1.0)
        c = np.cumsum(w)
        want.append(int(np.argmax(w)) if T[r] == 0 else int(np.searchsorted(c, np.float64(u[r]) * c[-1], side="right")))
    x, u, T = x.to(dev), u.to(dev), T.to(dev)
    tokens = torch.full((100, R), -7, dtype=torch.int32, device=dev)
    for out in tokens:
        q.sample(x, u, out, temperature=T)
    q.sync_status()
    assert (tokens.cpu() == torch.tensor(want, dtype=torch.int32)).all()


def weight_bounds(x, top, T):
    """2^42 exp((x - top) / T), below and above by what fp64's exponential (2^-52) and its argument (60 2^-53) leave open."""
    w = math.exp(float((Fraction(float(x)) - Fraction(float(top))) / Fraction(float(T)))) * 2.0 ** 42
    slack = Fraction(w * 2.0 ** -46)
    return Fraction(w) - slack, Fraction(w) + slack


def check_weights(dev, T, top, depths, seed=0):
    """A token's weight to one step of 2^-42, by whether the token is taken.

    Of three tokens (x, the largest, z) of weights w, 2^42 and t the first is
    taken where w > u (w + 2^42 + t).  For an fp32 u the logit z is the last
    one by whose weight the first token has to be taken, or the first by which
    it must not be, for every w and t less than 1 from their values."""
    T, top, rng = np.float32(T), np.float32(top), np.random.default_rng(seed)
    rows, want = [], []
    for depth in depths:
        x = np.float32(float(top) - depth * float(T))
        if not (x < top and np.isfinite(x)):
            continue
        lo, hi = weight_bounds(x, top, T)
        if lo < 8:
            continue
        # (a step of w moves the border by 1 / u - 1 of t, and u's own rounding by up to 2^19)
        t = 2.0 ** 20 * (1 + rng.random()) + 2.0 ** 44 / float(lo)
        u = np.float32(float(lo) / (float(lo) + 2.0 ** 42 + t))
        U = Fraction(float(u))
        sure = (lo - 1) * (1 - U) / U - 2 ** 42 - 1   # taken for all t up to this
        never = (hi + 1) * (1 - U) / U - 2 ** 42 + 1  # ... and not from this on
        for border, taken in ((sure, True), (never, False)):
            z = np.float32(float(top) + math.log(float(border) / 2.0 ** 42) * float(T))
            step = np.float32(-np.inf if taken else np.inf)
            while (weight_bounds(z, top, T)[1] > border) if taken else (weight_bounds(z, top, T)[0] < border):
                z = np.nextafter(z, step)
            rows.append((x, top, z, u)), want.append(taken)
    rows = torch.tensor(np.array(rows, np.float32))
    assert len(want) > 100
    tokens, _ = call(dev, rows[:, :3].contiguous().to(dev), rows[:, 3].contiguous().to(dev), T=float(T))
    q.sync_status()
    assert np.array_equal(tokens.cpu().numpy() == 0, np.array(want))


@pytest.mark.parametrize("T,top", [(1.0, 0.0), (1.0, 20.0), (0.7, -3.0), (1e-3, 0.5), (50.0, 100.0), (2e9, 1e9)])
def test_weights_are_off_by_less_than_their_step(dev, T, top):
    rng = np.random.default_rng(int(T * 10))
    check_weights(dev, T, top, np.concatenate((rng.uniform(0, 27, 800), rng.uniform(0, 2, 400), 10 ** rng.uniform(-6, 0, 100))))


@pytest.mark.parametrize("T,top", [(1e37, 3e38), (1e37, 0.0), (2e18, 1e18), (1e-37, 0.0), (1e-38, 1e-36), (1e-39, 0.0), (1e-42, 0.0),
                                   (5e-44, 1e-42), (1e-19, 1e-18), (9e-19, 0.0)])
def test_weights_of_temperatures_at_the_ends_of_fp32(dev, T, top):
    rng = np.random.default_rng(8)
    check_weights(dev, T, top, np.concatenate((rng.uniform(0, 27, 800), rng.uniform(0, 2, 400))))


@pytest.mark.parametrize("kw", [{}, dict(top_p=0.9), dict(top_k=900, top_p=0.9), dict(top_k=900, min_p=0.01)])
@pytest.mark.parametrize("T", [1e-44, 1e-40, 1e-30, 8e-19, 1e-18, 2e18, 1e30, 3e38])
def test_large_and_small_logits_at_any_temperature(dev, T, kw):
    """Logits that T tells apart, and such as lie far beyond what it does, of either sign."""
    z = logits_of(2500, seed=12).astype(np.float64)
    few = dict(most=50, T=T, **kw)
    x = np.clip(z * T, -3e38, 3e38)
    check(dev, x, **few)
    for far in (1e25, -1e25, 3e38, -1e38):
        if abs(far) < 1e6 * T:
            continue
        y = x.copy()
        y[::5] = far * (1 + np.arange(500) / 1000.0) if abs(far) < 1e38 else far
        if far < 0:
            y[1::5] = far
        check(dev, y, **few)
        check(dev, np.abs(y) * np.sign(far), **few)
