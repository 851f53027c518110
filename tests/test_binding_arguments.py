"""What the binding itself checks, on the host."""
import pytest
import torch

import int8_quantized_gb300 as q


def test_the_current_stream_initialises_cuda(monkeypatch):
    """Where CUDA cannot be initialised (a forked child, no driver) the call
    says what torch says, for every operator."""
    def refuse():
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")

    monkeypatch.setattr(torch.cuda, "_lazy_init", refuse)
    for call in (q._stream, q.sync_status, lambda: q.measure_int8_mma_peak(1)):
        with pytest.raises(RuntimeError, match="re-initialize CUDA"):
            call()


def test_a_torch_without_cuda_says_so(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)

    def refuse():
        raise AssertionError("Torch not compiled with CUDA enabled")

    monkeypatch.setattr(torch.cuda, "_lazy_init", refuse)
    with pytest.raises(AssertionError, match="not compiled with CUDA"):
        q._stream()


def test_q_out_without_q(monkeypatch):
    """It came back as it was, as if turned."""
    class Library:
        def __getattr__(self, name):
            return lambda *args: 0

    monkeypatch.setattr(q, "_L", lambda: Library())
    monkeypatch.setattr(q, "_page_table", lambda t, *a: q._lib.PageTableStruct())
    monkeypatch.setattr(q, "_rows", lambda *a: (None, 0, 0))
    monkeypatch.setattr(q, "_i32", lambda *a: None)
    monkeypatch.setattr(q, "_stream", lambda s=None: None)
    cache = type("Cache", (), {"_ref": None, "shape": (1, 1, 16, 64)})()
    k = torch.zeros((2, 1, 64))
    assert q.kv_append(cache, None, None, None, k, k) is None
    with pytest.raises(ValueError, match="q_out"):
        q.kv_append(cache, None, None, None, k, k, q_out=torch.zeros((2, 4, 64)))


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lies on a GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: self.where)


def on(t, where="cuda:0"):
    t = t.as_subclass(OnDevice)
    t.where = where
    return t


def pool(shape, dtype=torch.int8, where="cuda:0"):
    return on(torch.zeros(shape, dtype=dtype), where)


def test_cache_pools_lie_on_one_device():
    shape = (2, 2, 16, 64)
    scales = [pool(shape[:3], torch.float32) for _ in range(2)]
    q.KVCache(pool(shape), pool(shape), *scales)
    with pytest.raises(TypeError, match="v must be"):
        q.KVCache(pool(shape), pool(shape, where="cuda:1"), *scales)
    with pytest.raises(TypeError, match="v_scale must be"):
        q.KVCache(pool(shape), pool(shape), scales[0], pool(shape[:3], torch.float32, "cuda:1"))


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_cache_strides_of_one_place_mean_nothing(axis):
    """One page, one head or pages of one token: torch gives such an axis any
    stride, and differing ones to a view and to a copy."""
    shape = [3, 2, 16, 64]
    shape[axis] = 1
    strides = list(torch.zeros(shape).stride())
    strides[axis] = 5

    def view(dtype, n):
        return on(torch.zeros(1 << 14, dtype=dtype).as_strided(shape[:n], strides[:n] if n == 4 else
                                                              [s // 64 if i != axis else 3 for i, s in
                                                               enumerate(strides[:3])]))

    c = q.KVCache(view(torch.int8, 4), pool(shape), pool(shape[:3], torch.float32), view(torch.float32, 3),
                  pool(shape[:3], torch.float32))
    assert c.shape == tuple(shape)
    with pytest.raises(ValueError, match="shape and strides"):
        q.KVCache(pool(shape), on(torch.zeros([2 * n for n in shape], dtype=torch.int8)[tuple(slice(n) for n in shape)]),
                  pool(shape[:3], torch.float32), pool(shape[:3], torch.float32))


@pytest.mark.parametrize("one", ["pages", "kv_heads", "page_size"])
def test_the_library_takes_any_stride_of_one_place(one):
    import ctypes

    from int8_quantized_gb300 import _lib, build
    from test_kv_abi import cache, table
    build.build()
    lib = _lib.load()
    name = {"pages": "page_stride", "kv_heads": "head_stride", "page_size": "token_stride"}[one]
    for stride in (0, 5, -3):
        c = cache(**{one: 1, name: stride, "scale_" + name: stride})
        assert lib.i8q_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(table()), 4, 0) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("cache", ["s8", "bf16"])
def test_cache_with_an_axis_of_one_place(dev, axis, cache):
    """All four calls on pools whose axis of one place has an odd stride give what they give on contiguous ones."""
    g = torch.Generator()
    g.manual_seed(axis)
    shape = [40, 2, 16, 64]
    shape[axis] = 1
    if axis == 0:
        shape[2] = 128
    P, H, page, D = shape
    heads, length = 4 * H, min(36, 36 * page)
    dtype = torch.int8 if cache == "s8" else torch.bfloat16
    base = {n: torch.randint(-100, 100, shape, generator=g).to(dtype).to(dev) for n in ("k", "v")}
    per = {n: (torch.rand(shape[:3], generator=g) * 0.02 + 0.01).to(dev) for n in ("k_scale", "v_scale", "score")}
    if cache == "bf16":
        per = {"k_scale": None, "v_scale": None, "score": per["score"]}

    def odd(t):
        strides = list(t.stride())
        strides[axis] = 7
        return t.as_strided(t.shape, strides)

    results = []
    for change in (lambda t: t, odd):
        t = {n: None if x is None else change(x.clone()) for n, x in {**base, **per}.items()}
        c = q.KVCache(t["k"], t["v"], t["k_scale"], t["v_scale"], t["score"])
        h = torch.Generator()
        h.manual_seed(9)
        order = torch.randperm(P, generator=h).to(torch.int32).to(dev)
        table = order[None, :-(-length // page)].contiguous()
        x = torch.randn((3, heads + 2 * H, D), generator=h).to(dev)
        seq = torch.zeros(3, dtype=torch.int32, device=dev)
        index = torch.tensor([1, 9, length - 1], dtype=torch.int32, device=dev)
        lengths = torch.tensor([length], dtype=torch.int32, device=dev)
        q.kv_append(c, table, seq, index, x[:, heads:heads + H], x[:, heads + H:])
        out = torch.empty((1, heads, D), device=dev)
        q.paged_attention(c, table, lengths, x[:1, :heads], out, accumulate=True)
        back = [torch.empty((3, H, D), device=dev) for _ in range(2)]
        q.kv_gather(c, table, seq, index, *back)
        kept = torch.empty((1, H, 4), dtype=torch.int32, device=dev)
        if P > 1:
            q.kv_evict(c, table, lengths, order[None, -4:].contiguous(), kept, sink=1, recent=1)
        else:
            kept.zero_()
        results.append([out, *back, kept] + [x.clone() for x in t.values() if x is not None])
    q.sync_status()
    for a, b in zip(*results):
        assert torch.equal(a, b)
