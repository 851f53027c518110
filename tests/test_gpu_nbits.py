"""MatMulNBits on a GB300 against the definition in 64 bits.

Tolerances, with a = sum_k |A| |q - z| |s| of an output: a block's products are
exact in 22 bits at most and summed by the tensor pipe, which cuts what falls
below 2^-23 of the largest term of a step of 16 (and of the sum so far), twice
that at most: 2^-22 a for each of the up to 8 steps of a block; the fma of each
block and the sums over warps and clusters round by 2^-24 of a sum that is at
most a: (K / block + 32) 2^-24 a.  (fp32 activations: three products a step, so
three cuts, each step then rounded: (K / 16 + 32) 2^-24 a.)  The bias adds one
rounding, the output half a step of its type."""
import pytest
import torch

import int8_quantized_gb300 as q

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def weights(g, N, K, block, scales="bf16", zero=True):
    blocks = -(-K // block)
    B = torch.randint(0, 256, (N, blocks, block // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    s = ((torch.rand((N, blocks), generator=g) + 0.1) * 0.1 * torch.randint(-1, 2, (N, blocks), generator=g)).to(TYPES[scales])
    z = torch.randint(0, 256, (N, -(-blocks // 2)), generator=g, dtype=torch.int64).to(torch.uint8) if zero else None
    return B, s, z


def dense(B, s, z, K, block):
    """q - z and s, fp64 [N, K]."""
    N, blocks = s.shape
    c = torch.stack((B & 15, B >> 4), -1).view(N, -1).double()
    zp = torch.full((N, blocks), 8.0, dtype=torch.float64) if z is None else torch.stack((z & 15, z >> 4), -1).view(
        N, -1)[:, :blocks].double()
    return (c - zp.repeat_interleave(block, 1))[:, :K], s.double().repeat_interleave(block, 1)[:, :K]


def tolerance(size, want, K, block, type, bias):
    if type == "f32":
        sums = 3 * 2.0 ** -22 + (K / 16 + 32) * 2.0 ** -24
    else:
        sums = 8 * 2.0 ** -22 + (K / min(block, 128) + 32) * 2.0 ** -24
    tol = sums * size + (2.0 ** -24 * want.abs() if bias is not None else 0)
    return tol * 1.01 + (2.0 ** -8 if type == "bf16" else 2.0 ** -24) * want.abs() + 1e-37


def check(dev, M, N, K, block, type="bf16", scales="bf16", zero=True, bias=False, seed=0, pad=0, offset=0, gain=1.0):
    g = gen(seed)
    B, s, z = weights(g, N, K, block, scales, zero)
    b = torch.randn((N,), generator=g) if bias else None
    A = (torch.randn((M, K), generator=g) * gain)
    A[:, ::17] *= 30
    A = A.to(TYPES[type])
    up = lambda t: None if t is None else t.to(dev)
    m = q.MatMulNBits(up(B), up(s), K, block, zero_points=up(z), bias=up(b))
    rows = torch.zeros((M, K + pad + offset), dtype=A.dtype, device=dev)[:, offset:offset + K]
    rows.copy_(A)
    wide = torch.full((M + 1, N + pad + offset), 9.0, dtype=A.dtype, device=dev)
    Y = wide[:M, offset:offset + N]
    assert m.forward(rows, Y) is Y
    q.sync_status()
    w, sc = dense(B, s, z, K, block)
    want = A.double() @ (w * sc).t() + (0 if b is None else b.double())
    size = A.double().abs() @ (w * sc).abs().t()
    got = Y.cpu().double()
    tol = tolerance(size, want, K, block, type, b)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
    wide[:M, offset:offset + N] = 9.0
    assert (wide == 9.0).all()  # nothing beside the rows is written


@pytest.mark.parametrize("block", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("type,scales,zero", [("bf16", "bf16", True), ("bf16", "f32", False), ("f32", "f32", True),
                                              ("f32", "bf16", False)])
def test_blocks_and_types(dev, block, type, scales, zero):
    check(dev, 3, 70, 1000, block, type, scales, zero, bias=zero, seed=block)
    check(dev, 1, 33, 4096, block, type, scales, zero, seed=block)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_rows(dev, M, type):
    check(dev, M, 100, 640, 32, type, seed=M)
    check(dev, M, 50, 2500, 128, type, zero=False, seed=M)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 33, 2433, 5000])
def test_outputs(dev, N):
    check(dev, 5, N, 384, 32, seed=N)
    check(dev, 20, N, 130, 64, bias=True, seed=N)


@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 31, 127, 128, 129, 255, 257, 2047, 2049, 4097, 8192, 8200])
@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_depths(dev, K, type):
    check(dev, 4, 40, K, 32, type, seed=K)
    check(dev, 12, 20, K, 256, type, seed=K)


@pytest.mark.parametrize("M", [1, 12, 40])
@pytest.mark.parametrize("K", [14336, 16384, 33000, 70000])
@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_deep_products_by_clusters(dev, M, K, type):
    check(dev, M, 60, K, 64, type, seed=K)


@pytest.mark.parametrize("M", [9, 16, 17, 33, 64, 65, 200])
@pytest.mark.parametrize("N,K,block", [(128, 128, 128), (100, 200, 16), (1000, 384, 32), (3000, 640, 64), (20000, 384, 128),
                                       (2433, 4096, 32), (500, 14336, 64), (130, 33000, 128), (40, 70000, 256)])
def test_many_rows(dev, M, N, K, block):
    """The tcgen05 kernel: 16, 32 and 64 rows at a time, each block, odd and even numbers of chunks a CTA,
    activations that stay and that are sent for again, clusters of each size."""
    check(dev, M, N, K, block, scales="f32" if M % 2 else "bf16", zero=block != 64, bias=M == 33, seed=M)


def test_many_rows_unaligned(dev):
    check(dev, 20, 300, 1000, 32, pad=1)
    check(dev, 20, 300, 1000, 32, offset=3, pad=5)
    check(dev, 20, 300, 1000, 32, pad=8)


def test_many_strips_of_a_cluster(dev):
    """More groups of strips than a cluster joins at once."""
    check(dev, 3, 16 * 700, 14336, 128, seed=1)
    check(dev, 3, 16 * 700, 4096, 128, "f32", seed=2)


@pytest.mark.parametrize("type", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (1, 0), (0, 1), (3, 2), (4, 4)])
def test_strides_and_alignment(dev, type, pad, offset):
    check(dev, 5, 37, 300, 32, type, pad=pad, offset=offset)
    check(dev, 1, 37, 301, 16, type, pad=pad, offset=offset)


def test_large_and_small_activations(dev):
    check(dev, 4, 64, 512, 32, "f32", gain=1e30)
    check(dev, 4, 64, 512, 32, "f32", gain=1e-30)
    check(dev, 4, 64, 512, 32, "bf16", gain=1e-30)


@pytest.mark.parametrize("type", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("R", [3, 20])
def test_a_row_that_is_not_finite_stays_alone(dev, R, type, bad):
    g = gen(3)
    N, K, block = 40, 256, 32
    B, s, z = weights(g, N, K, block, "f32", False)
    s = s.abs() + 0.01
    rows = [0] + list(range(2, R))
    A = torch.randn((R, K), generator=g)
    A[1, 77] = bad
    A = A.to(TYPES[type])
    m = q.MatMulNBits(B.to(dev), s.to(dev), K, block)
    Y = torch.empty((R, N), dtype=A.dtype, device=dev)
    m.forward(A.to(dev), Y)
    q.sync_status()
    w, sc = dense(B, s, None, K, block)
    y = Y.cpu().float()
    assert torch.isfinite(y[rows]).all()
    c = w[:, 77]
    if bad != bad:
        assert torch.isnan(y[1]).all()
    else:  # infinity times the code: its sign, or NaN for a code of 0
        assert torch.isnan(y[1][c == 0]).all()
        assert (y[1][c != 0] == (torch.sign(c[c != 0]) * bad).float()).all()


def test_largest_finite_activation_is_not_an_infinity(dev):
    B = torch.full((16, 1, 8), 0x98, dtype=torch.uint8, device=dev)  # codes 0 and 1
    m = q.MatMulNBits(B, torch.full((16, 1), 0.5, device=dev), 16, 16)
    A = torch.zeros((1, 16), device=dev)
    A[0, 1] = torch.finfo(torch.float32).max
    Y = torch.empty((1, 16), device=dev)
    m.forward(A, Y)
    assert (Y == torch.finfo(torch.float32).max / 2).all()


def test_values_near_each_other_cancel_exactly(dev):
    """Sums that cancel: what remains is the small terms', to the bit."""
    K = 512
    A = torch.zeros((1, K))
    A[0, :256], A[0, 256:512] = 1.0, -1.0
    A[0, 511] = 0.0
    B = torch.full((16, K // 32, 16), 0xFF, dtype=torch.uint8)
    m = q.MatMulNBits(B.to(dev), torch.full((16, K // 32), 3.0, device=dev), K, 32)
    Y = torch.empty((1, 16), device=dev)
    m.forward(A.to(dev), Y)
    assert (Y == 21.0).all()


def test_codes_at_an_odd_address(dev):
    g = torch.Generator()
    g.manual_seed(4)
    B, s, z = weights(g, 50, 300, 32)
    odd = torch.empty(B.numel() + 1, dtype=torch.uint8, device=dev)[1:]
    odd.copy_(B.flatten())
    a, b = (q.MatMulNBits(t, s.to(dev), 300, 32, zero_points=z.to(dev)) for t in (odd.view(B.shape), B.to(dev)))
    assert torch.equal(a.packed, b.packed)


def test_no_rows(dev):
    B, s, z = weights(gen(0), 20, 64, 32)
    m = q.MatMulNBits(B.to(dev), s.to(dev), 64, 32, zero_points=z.to(dev))
    m.forward(torch.empty((0, 64), device=dev), torch.empty((0, 20), device=dev))
    q.sync_status()


@pytest.mark.parametrize("rows", [3, 9, 50])
def test_repeats_streams_and_graphs(dev, rows):
    g = gen(5)
    N, K = 300, 14336
    B, s, z = (t.to(dev) for t in weights(g, N, K, 32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m = q.MatMulNBits(B, s, K, 32, zero_points=z, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    B.fill_(0), s.fill_(0), z.fill_(0)  # not read again
    A = torch.randn((rows, K), generator=g).to(torch.bfloat16).to(dev)
    one, two, three = (torch.empty((rows, N), dtype=torch.bfloat16, device=dev) for _ in range(3))
    m.forward(A, one)
    m.forward(A, two)
    side.wait_stream(torch.cuda.current_stream())
    m.forward(A, three, stream=side)
    torch.cuda.synchronize()
    assert one.abs().sum() > 0 and torch.equal(one, two) and torch.equal(one, three)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for gr in (graph, other):
        with torch.cuda.graph(gr):
            m.forward(A, three)
    three.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(one, three)
    A.mul_(2.0)
    other.replay()
    torch.cuda.synchronize()
    assert torch.equal((one.float() * 2).to(torch.bfloat16), three)


def test_refusals(dev):
    B, s, z = (t.to(dev) for t in weights(gen(0), 20, 64, 32))
    for bad, match in ((dict(B=B.view(torch.int8)), "B must be"), (dict(B=B[:, :1]), "B must be"), (dict(scales=s[:, :1]), "scales must"),
                       (dict(zero_points=z[:10]), "zero_points must"), (dict(bias=s[0]), "bias must")):
        kw = dict(B=B, scales=s, K=64, block_size=32, zero_points=z)
        kw.update(bad)
        with pytest.raises(ValueError, match=match):
            q.MatMulNBits(**kw)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        q.MatMulNBits(B, s.half(), 64, 32)
    with pytest.raises(TypeError, match="CUDA"):
        q.MatMulNBits(B.cpu(), s, 64, 32)
    with pytest.raises(q.I8QError, match="block_size"):
        q.MatMulNBits(B.view(20, 16, 2), torch.ones((20, 16), device=dev), 64, 4)
    m = q.MatMulNBits(B, s, 64, 32, zero_points=z)
    A, Y = torch.ones((3, 64), device=dev), torch.full((3, 20), 5.0, device=dev)
    for a, y, err, match in ((A[:, :63], Y, ValueError, "A must be"), (A, Y[:2], ValueError, "A must be"),
                             (A, Y.to(torch.bfloat16), TypeError, "one dtype"), (A.half(), Y.half(), TypeError, "float32"),
                             (A.cpu(), Y, TypeError, "tensors on"), (A.t().contiguous().t(), Y, ValueError, "contiguous"),
                             (A[:1].expand(3, 64), Y, q.I8QError, "overlap"), (A, Y[:1].expand(3, 20), q.I8QError, "overlap")):
        with pytest.raises(err, match=match):
            m.forward(a, y)
    torch.cuda.synchronize()
    assert (Y == 5.0).all()


def products(dev, A, B, s, z, K, block, bias=None):
    """Y and, in 64 bits, what it should be and the sum of its terms' sizes."""
    up = lambda t: None if t is None else t.to(dev)
    m = q.MatMulNBits(up(B), up(s), K, block, zero_points=up(z), bias=up(bias))
    Y = torch.empty((A.shape[0], B.shape[0]), dtype=A.dtype, device=dev)
    m.forward(A.to(dev), Y)
    q.sync_status()
    w, sc = dense(B, s, z, K, block)
    want = A.double() @ (w * sc).t() + (0 if bias is None else bias.double())
    return Y.cpu().double(), want, A.double().abs() @ (w * sc).abs().t()


@pytest.mark.parametrize("M", [1, 8, 9, 40, 70])
@pytest.mark.parametrize("block", [16, 128, 256])
@pytest.mark.parametrize("type,scales", [("bf16", "bf16"), ("f32", "f32")])
def test_products_beyond_fp32_before_their_scale(dev, M, block, type, scales):
    """Activations as large as the type has them: a block's products pass fp32's range, Y does not."""
    g = gen(M)
    N, K = 70, 700
    B, s, z = weights(g, N, K, block, scales)
    A = ((torch.rand((M, K), generator=g) * 0.5 + 0.5) * torch.randint(0, 2, (M, K), generator=g).mul(2).sub(1))
    A = (A.double() * torch.finfo(TYPES[type]).max).to(TYPES[type])
    A[0] = torch.finfo(TYPES[type]).max
    bias = torch.randn((N,), generator=g) * 1e33
    s = (s.float() * 2.0 ** -12).to(s.dtype)
    got, want, size = products(dev, A, B, s, z, K, block, bias)
    assert want.abs().max() < 3e38 and torch.isfinite(A).all()
    tol = tolerance(size, want, K, block, type, bias)
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("share", [1.0, 0.5])
@pytest.mark.parametrize("M", [2, 20])
@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_a_sum_beyond_fp32_on_its_way(dev, M, type, share):
    K, block = 256, 32
    B = torch.full((16, K // block, block // 2), 0xFF, dtype=torch.uint8)  # 7 after the zero point
    B[:, 4:] = 0x11                                                       # -7
    B[:, 7, 0] = 0x12                                                     # and one of -6
    A = torch.full((M, K), torch.finfo(TYPES[type]).max * share).to(TYPES[type])
    got, want, size = products(dev, A, B, torch.ones((16, K // block)), None, K, block)
    assert (want == A[0, 0].double()).all()
    tol = tolerance(size, want, K, block, type, None)
    # (the tolerance is that of the sum before its rounding to the type: Y = fp32's largest number, plus a part of the
    # 1792 times as large sum of the terms' sizes, may round to an infinity; half of it, off by 0.007 of it, may not)
    beyond = torch.isposinf(got) & (want + tol > torch.finfo(torch.float32).max)
    assert not beyond.any() or (type, share) == ("f32", 1.0)
    assert ((got - want).abs().le(tol) | beyond).all()


@pytest.mark.parametrize("M", [3, 20])
@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_smallest_activations_and_largest_scales(dev, M, type):
    """Subnormal activations, whole multiples of 2^-133, by scales of 2^90; what of a row's sum lies below 2^-137 (of
    its blocks' and warps' parts: (K / 16 + 32) of them) is lost."""
    g = gen(M)
    N, K, block = 40, 400, 32
    B, s, z = weights(g, N, K, block, "f32")
    A = torch.randint(-3000, 3001, (M, K), generator=g).double() * 2.0 ** -133
    A = A.to(TYPES[type])
    got, want, size = products(dev, A, B, s * 2.0 ** 90, z, K, block)
    assert want.abs().max() > 0 and ((got - want).abs() <= tolerance(size, want, K, block, type, None)).all()
    got, want, size = products(dev, A, B, s, z, K, block)
    tol = tolerance(size, want, K, block, type, None) - 1e-37 + (K / 16 + 32) * 2.0 ** -137
    assert ((got - want).abs() <= tol + (2.0 ** -133 if type == "bf16" else 2.0 ** -149)).all()


@pytest.mark.parametrize("type,M,K,ctas,rounds", [("f32", 3, 4096, 2, 17), ("f32", 40, 4096, 2, 33), ("bf16", 40, 14336, 2, 17),
                                                  ("bf16", 20, 14336, 2, 35), ("bf16", 30, 33000, 8, 18), ("f32", 24, 33000, 8, 33),
                                                  ("bf16", 33, 70000, 8, 17)])
def test_more_strips_than_a_cluster_joins_at_once(dev, type, M, K, ctas, rounds):
    """A cluster's CTAs hold the sums of 16 groups of strips between two
    meetings; these have 17 to 35, so that what they hold is written anew.
    (Rows of bf16 at an odd place go 8 at a time, as fp32's do, and each 8 have
    a share of the clusters.)"""
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    clusters = sms // ctas // -(-M // 8)
    check(dev, M, 16 * ((rounds - 1) * clusters + clusters // 2 + 1) - 3, K, 128, type, offset=1, pad=2, seed=rounds)
