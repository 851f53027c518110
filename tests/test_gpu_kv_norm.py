"""kv_append with norms of the heads of q and k.  Every operation after the sum
of squares rounds once, so the call gives, bit for bit, what the call without
norms gives for rows normalized beforehand in fp32 (numpy; the mean of squares
from fp64, rounded once).  And by the formula in 64 bits: the mean is off by
half a step (2^-25 of the root), eps' sum, the root, the reciprocal and two
products by one rounding each, 5 2^-24 together; the rotation's three
roundings act on |x1| + |x2|."""
import numpy as np
import pytest
import torch

import int8_quantized_gb300 as q
from test_gpu_kv_cache import TYPES, gen, make_cache, make_table

pytestmark = pytest.mark.gpu


def normed(x, w, eps):
    """x fp32 [..., D], w fp32 [D], as the definition rounds."""
    x = x.numpy()
    with np.errstate(all="ignore"):
        mean = ((x.astype(np.float64) ** 2).sum(-1, keepdims=True) / x.shape[-1]).astype(np.float32)
        inverse = np.float32(1) / np.sqrt(mean + np.float32(eps))
        y = (x * inverse) * w.numpy()
    assert y.dtype == np.float32
    return torch.from_numpy(y)


def setup(dev, T, Hq, H, D, page, type, cache, rot, axes=1, seed=0, edit=None, weights=torch.float32, order="phtd"):
    g = gen(seed)
    table, pages, _ = make_table(g, dev, [T], page)
    c, d = (make_cache(gen(seed + 1), dev, pages, H, page, D, cache, order) for _ in range(2))
    x = torch.randn((T, Hq + 2 * H, D), generator=g) * (torch.rand((T, 1, 1), generator=g) * 5 + 0.01)
    if edit:
        edit(x)
    x = x.to(TYPES[type])
    w = [(torch.randn((D,), generator=g) * 0.3 + 1).to(weights) for _ in range(2)]
    kw = {}
    if rot:
        ang = torch.rand((70, rot // 2), generator=g, dtype=torch.float64) * 6.28
        kw = dict(positions=torch.randint(0, 70, (axes, T), generator=g).to(torch.int32).to(dev),
                  cos=ang.cos().float().to(dev), sin=ang.sin().float().to(dev),
                  pair_axis=[j % axes for j in range(rot // 2)])
    seq, index = torch.zeros(T, dtype=torch.int32, device=dev), torch.arange(T, dtype=torch.int32, device=dev)
    return table, c, d, x, w, kw, seq, index


def check(dev, T, Hq, H, D, page, type, cache, rot=0, axes=1, seed=0, which="qk", eps=1e-6, edit=None, strided=False,
          inplace=False, weights=torch.float32, order="phtd", interleaved=False):
    table, c, d, x, w, kw, seq, index = setup(dev, T, Hq, H, D, page, type, cache, rot, axes, seed, edit, weights, order)
    if rot:
        kw["interleaved"] = interleaved
    parts = x.float().split((Hq, H, H), 1)
    ready = [normed(p, v.float(), eps) if n in which else p for p, v, n in zip(parts, w, "qk")] + [parts[2]]
    want_q = torch.empty((T, Hq, D), device=dev) if Hq else None
    qx = dict(q=ready[0].to(dev), q_out=want_q) if Hq else {}
    q.kv_append(d, table, seq, index, ready[1].to(dev), ready[2].to(dev), **qx, **kw)
    rows = x.to(dev)
    if strided:  # rows that begin at odd places
        wide = torch.zeros((T, Hq + 2 * H, D + 3), dtype=x.dtype, device=dev)
        wide[..., 3:] = rows
        rows = wide[..., 3:]
    xq, xk, xv = rows.split((Hq, H, H), 1)
    got_q = None
    if Hq:
        got_q = xq if inplace else torch.empty((T, Hq, D), dtype=x.dtype, device=dev)
        kw.update(q=xq, q_out=got_q)
    kw.update({n + "_norm": v.to(dev) for n, v in zip("qk", w) if n in which})
    q.kv_append(c, table, seq, index, xk, xv, norm_eps=eps, **kw)
    q.sync_status()
    for n in ("k", "v", "k_scale", "v_scale", "score"):
        a, b = getattr(c, n), getattr(d, n)
        if a is not None:
            a, b = ((t.cpu() if t.dtype == torch.int8 else torch.nan_to_num(t.cpu().float(), nan=123.0)) for t in (a, b))
            assert torch.equal(a, b), n
    if Hq:
        a, b = torch.nan_to_num(got_q.cpu().float(), nan=123.0), torch.nan_to_num(want_q.to(x.dtype).cpu().float(), nan=123.0)
        assert torch.equal(a, b)


@pytest.mark.parametrize("type", ["bf16", "f32"])
@pytest.mark.parametrize("cache", ["s8", "bf16"])
@pytest.mark.parametrize("D,rot", [(16, 16), (64, 32), (80, 80), (96, 0), (128, 128), (144, 8), (192, 64), (256, 256)])
def test_heads_as_normalized_beforehand(dev, D, rot, type, cache):
    check(dev, 23, 6, 2, D, 16, type, cache, rot, seed=D)
    check(dev, 5, 6, 2, D, 16, type, cache, rot, seed=D, strided=True, interleaved=True, weights=torch.bfloat16)


@pytest.mark.parametrize("T,Hq,H", [(1, 1, 1), (1, 32, 8), (3, 71, 1), (300, 12, 12), (2500, 8, 2), (17, 0, 3)])
def test_tokens_and_heads(dev, T, Hq, H):
    check(dev, T, Hq, H, 128, 16, "bf16", "s8", 128, 3, seed=T, which="qk" if Hq else "k")
    check(dev, T, Hq, H, 64, 5, "f32", "bf16", 30, 2, seed=T, which="qk" if Hq else "k")


@pytest.mark.parametrize("which", ["q", "k", "qk"])
@pytest.mark.parametrize("strided", [False, True])
def test_one_norm_or_both_and_in_place(dev, which, strided):
    check(dev, 40, 8, 2, 128, 16, "bf16", "s8", 64, which=which, strided=strided, order="pthd", inplace=True)
    check(dev, 40, 8, 2, 80, 16, "f32", "bf16", 80, which=which, strided=strided, order="tphd", interleaved=True,
          inplace=True)


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("D", [64, 96, 256])
def test_extreme_rows(dev, strided, D):
    """Zero, subnormal and huge rows (whose squares fp32 does not hold), one large element, infinities and NaN."""
    def edit(x):
        x[0] = 0
        x[1] = 1e-42
        x[2] = 0
        x[2, :, 5] = -3.0
        x[3] *= 1e36
        x[4] *= 1e-30
        x[5] = 2.5e38
        x[6, :, 7] = float("inf")
        x[7, :, 8] = float("nan")
        x[8, :, 3] = 1e19
        x[9] *= 1e-8
    for eps in (1e-6, 0.0, 1.0):
        check(dev, 12, 4, 2, D, 16, "f32", "bf16", 64, edit=edit, strided=strided, eps=eps)
        check(dev, 12, 4, 2, D, 16, "bf16", "bf16", 64, edit=edit, strided=strided, eps=eps)

    def finite(x):  # (codes of rows that are not finite have no definition)
        edit(x)
        x[6], x[7] = 1.0, 2.0
        x[5] = 2.5e17
    check(dev, 12, 4, 2, D, 16, "f32", "s8", 64, edit=finite, strided=strided)


@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_against_the_formula_in_64_bits(dev, type):
    T, Hq, H, D = 50, 8, 2, 128
    table, c, _, x, w, kw, seq, index = setup(dev, T, Hq, H, D, 16, type, "bf16", 128, seed=9)
    out = torch.empty((T, Hq, D), dtype=x.dtype, device=dev)
    q.kv_append(c, table, seq, index, *x.to(dev)[:, Hq:].split((H, H), 1), q=x.to(dev)[:, :Hq], q_out=out,
                q_norm=w[0].to(dev), k_norm=w[1].to(dev), norm_eps=1e-5, **kw)
    q.sync_status()
    y = x[:, :Hq].double()
    y = y / (y.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w[0].double()
    pos = kw["positions"][0].cpu().long()
    cos, sin = kw["cos"].cpu().double()[pos][:, None], kw["sin"].cpu().double()[pos][:, None]
    a, b = y[..., :64], y[..., 64:]
    want = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    tol = 8 * 2.0 ** -24 * size + (2.0 ** -8 if type == "bf16" else 0) * want.abs()
    assert (torch.abs(out.cpu().double() - want) <= tol).all()


def test_refusals(dev):
    table, c, _, x, w, kw, seq, index = setup(dev, 4, 2, 1, 64, 16, "f32", "bf16", 0)
    xq, xk, xv = x.to(dev).split((2, 1, 1), 1)
    out, good = torch.full((4, 2, 64), 5.0, device=dev), w[0].to(dev)
    before = c.k.clone()

    def call(**kw):
        q.kv_append(c, table, seq, index, xk, xv, q=xq, q_out=out, **kw)

    with pytest.raises(ValueError, match="q_norm must be"):
        call(q_norm=good[:32])
    with pytest.raises(ValueError, match="k_norm must be"):
        call(k_norm=good[None])
    with pytest.raises(TypeError, match="CUDA"):
        call(q_norm=w[0])
    with pytest.raises(TypeError, match="one dtype"):
        call(q_norm=good, k_norm=good.to(torch.bfloat16))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        call(k_norm=good.half())
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(q.I8QError, match="eps"):
            call(k_norm=good, norm_eps=eps)
    with pytest.raises(ValueError, match="q_norm need"):
        q.kv_append(c, table, seq, index, xk, xv, q_norm=good)
    torch.cuda.synchronize()
    assert torch.equal(c.k, before) and (out == 5.0).all()


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 112, 128, 144, 192])
def test_a_key_that_is_not_finite_leaves_its_value_alone(dev, D, strided, type):
    """Where a row has fewer elements than its lanes hold, the lanes past its
    end take the norm's factor too: an infinity (a zero row, eps 0) or a NaN.
    The values' codes and scales are those of the call without norms."""
    T, Hq, H = 20, 4, 2
    g = gen(D)
    table, pages, _ = make_table(g, dev, [T], 16)
    c, d = (make_cache(gen(7), dev, pages, H, 16, D, "s8") for _ in range(2))
    x = torch.randn((T, Hq + 2 * H, D), generator=g)
    x[0, :-H] = 0.0
    x[1, :-H, 3] = float("nan")
    x[2, :-H, D - 1] = float("inf")
    x[3, :-H] = 1e-30
    x[4] = 0.0
    x = x.to(TYPES[type])
    rows = torch.zeros((T, Hq + 2 * H, D + 3 * strided), dtype=x.dtype, device=dev)[..., 3 * strided:]
    rows.copy_(x)
    xq, xk, xv = rows.split((Hq, H, H), 1)
    w = torch.full((D,), 0.5, device=dev)
    seq, index = torch.zeros(T, dtype=torch.int32, device=dev), torch.arange(T, dtype=torch.int32, device=dev)
    out = torch.empty((T, Hq, D), dtype=x.dtype, device=dev)
    for which in (dict(k_norm=w), dict(q_norm=w, k_norm=w)):
        q.kv_append(c, table, seq, index, xk, xv, q=xq, q_out=out, norm_eps=0.0, **which)
        q.kv_append(d, table, seq, index, xk, xv, q=xq, q_out=torch.empty_like(out))
        q.sync_status()
        assert torch.isfinite(c.v_scale).all()
        assert torch.equal(c.v, d.v) and torch.equal(c.v_scale, d.v_scale)
        k_back, v_back = (torch.empty((T, H, D), device=dev) for _ in range(2))
        q.kv_gather(c, table, seq, index, k_back, v_back)
        most = x[:, -H:].float().abs().amax(-1, keepdim=True)
        assert ((v_back.cpu() - x[:, -H:].float()).abs() <= 0.501 / 127 * most).all()
        assert torch.isnan(k_back[1]).all()
