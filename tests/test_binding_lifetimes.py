"""What a MatMulNBits reads on a stream is recorded there, so that torch's
allocator does not hand its memory on before it has been read.  On the host
with the library and the streams replaced; on a GPU with work queued before
the calls, and the freed memory overwritten at once."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

import int8_quantized_gb300 as q
from test_binding_arguments import OnDevice


class Recording(OnDevice):
    """A CPU tensor that says it lies on a GPU, and notes the streams that read it."""

    def record_stream(self, stream):
        self.streams.append(stream)


def recording(t):
    t = t.as_subclass(Recording)
    t.where, t.streams = torch.device("cuda:0"), []
    return t


@pytest.fixture
def host(monkeypatch):
    class Library:
        def __getattr__(self, name):
            return lambda *args: 4096 if name.endswith("_size") else 0

    state = SimpleNamespace(current=SimpleNamespace(cuda_stream=3), allocated=[])

    def workspace(size, device, stream):
        state.allocated.append(recording(torch.zeros(size, dtype=torch.uint8)))
        return state.allocated[-1]

    monkeypatch.setattr(q, "_L", lambda: Library())
    monkeypatch.setattr(q, "_workspace", workspace)
    monkeypatch.setattr(q, "_stream", lambda s=None: ctypes.c_void_p((s or state.current).cuda_stream))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state.current)
    return state


def make(stream=None, bias=True):
    t = [recording(torch.zeros((16, 2, 16), dtype=torch.uint8)), recording(torch.zeros((16, 2))),
         recording(torch.zeros((16, 1), dtype=torch.uint8)), recording(torch.zeros(16)) if bias else None]
    return q.MatMulNBits(t[0], t[1], 64, 32, zero_points=t[2], bias=t[3], stream=stream), t


@pytest.mark.parametrize("given", [False, True])
def test_the_layout_reads_on_its_stream(host, given):
    side = SimpleNamespace(cuda_stream=7)
    _, t = make(side if given else None)
    for x in t[:3]:
        assert x.streams == [side if given else host.current]


@pytest.mark.parametrize("bias", [False, True])
def test_calls_read_on_theirs(host, bias):
    home, side, other = host.current, SimpleNamespace(cuda_stream=7), SimpleNamespace(cuda_stream=0)
    m, t = make(bias=bias)
    read = [m.packed] + [t[3]] * bias
    A, Y = recording(torch.zeros((2, 64))), recording(torch.zeros((2, 16)))
    before = [len(x.streams) for x in read]
    for stream, current in ((None, home), (side, home), (None, other), (side, home), (None, home), (None, other), (other, home)):
        host.current = current
        m.forward(A, Y, stream=stream)
    for x, n in zip(read, before):
        assert x.streams[n:] == [home, side, other]


def matrix(N, K, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randint(0, 256, (N, K // 32, 16), generator=g, dtype=torch.int64).to(torch.uint8),
            torch.rand((N, K // 32), generator=g) + 0.5,
            torch.randint(0, 256, (N, K // 64), generator=g, dtype=torch.int64).to(torch.uint8), torch.randn((N,), generator=g))


def occupy(dev, stream, work):
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(20):
            torch.mm(work, work)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["argument", "current"])
def test_what_a_busy_stream_still_has_to_read(dev, form):
    N, K = 512, 1024
    cpu = matrix(N, K)
    A = torch.randn((3, K)).to(dev)
    ready = q.MatMulNBits(*(t.to(dev) for t in cpu[:2]), K, 32, zero_points=cpu[2].to(dev), bias=cpu[3].to(dev))
    want, Y = (torch.empty((3, N), device=dev) for _ in range(2))
    ready.forward(A, want)
    side, work = torch.cuda.Stream(), torch.ones((4096, 4096), device=dev)
    for _ in range(3):
        # the layout: its inputs dropped at once, and written over on the current stream
        B, s, z, b = (t.to(dev) for t in cpu)
        occupy(dev, side, work)
        if form == "argument":
            m = q.MatMulNBits(B, s, K, 32, zero_points=z, bias=b, stream=side)
        else:
            with torch.cuda.stream(side):
                m = q.MatMulNBits(B, s, K, 32, zero_points=z, bias=b)
        shapes = [(t.shape, t.dtype) for t in (B, s, z)]
        del B, s, z
        over = [torch.full(n, 77, dtype=d, device=dev) for n, d in shapes]
        torch.cuda.synchronize()
        m.forward(A, Y)
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
        # a call: the handle and the bias dropped at once
        Y.zero_()
        m = q.MatMulNBits(*(t.to(dev) for t in cpu[:2]), K, 32, zero_points=cpu[2].to(dev), bias=cpu[3].to(dev))
        occupy(dev, side, work)
        if form == "argument":
            m.forward(A, Y, stream=side)
        else:
            with torch.cuda.stream(side):
                m.forward(A, Y)
        size = m.packed.numel()
        del m, b
        over += [torch.full((size,), 77, dtype=torch.uint8, device=dev), torch.full((N,), 77.0, device=dev),
                 torch.full((N,), 77.0, device=dev)]
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
        del over
