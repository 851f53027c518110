"""Scratch memory that the binding allocates for a call on another stream
belongs to that stream.  A block of the current stream's may still be in use
there (freed on the host, its work queued), and the call would write it at
once.  Shown on the host with the library, the allocator and the stream
context replaced; on a GPU the same calls give the results they should."""
import contextlib

import pytest
import torch

import int8_quantized_gb300 as q


class Library:
    """Every entry point: sizes 4096, status 0."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("_size") else 0


class Side:
    cuda_stream = 7
    device = "side's device"


@pytest.fixture
def allocations(monkeypatch):
    """(size, stream that was current) of each allocation."""
    current, seen, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    def recorded(*args, **kw):
        seen.append((args[0], current[0]))
        t = empty(args[0], dtype=kw["dtype"])
        t.record_stream = lambda s: None
        return t

    monkeypatch.setattr(q, "_L", lambda: Library())
    monkeypatch.setattr(q, "_dev", lambda t, *a: None)
    monkeypatch.setattr(q, "_stream", lambda s=None: None)
    monkeypatch.setattr(q, "_page_table", lambda t, *a: q._lib.PageTableStruct())
    monkeypatch.setattr(q, "_rows", lambda *a: (None, 0, 0))
    monkeypatch.setattr(q, "_i32", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    return seen


def calls():
    a, b, y = torch.zeros((4, 8), dtype=torch.uint8), torch.zeros((8, 4), dtype=torch.int8), torch.zeros((4, 4))
    one, f = torch.ones(1), torch.zeros((4, 8))
    x, w = torch.zeros((1, 1, 4, 4), dtype=torch.uint8), torch.zeros((1, 1, 3, 3), dtype=torch.int8)
    z = torch.zeros(1, dtype=torch.int8)
    cache = type("Cache", (), {"_ref": None, "shape": (1, 1, 16, 64)})()
    qx = torch.zeros((1, 2, 64))
    return {
        "qlinearconv": lambda s: q.qlinearconv(x, 1.0, 0, w, one, z, 1.0, 0, x, stream=s),
        "qgemm": lambda s: q.qgemm(a, 1.0, 0, b, one, y, stream=s),
        "matmul_integer_to_float": lambda s: q.matmul_integer_to_float(a, b, one, one, y, stream=s),
        "dynamic_quantize_matmul": lambda s: q.dynamic_quantize_matmul(f, b, one, y, stream=s),
        "paged_attention": lambda s: q.paged_attention(cache, torch.zeros((1, 1)), None, qx, qx, stream=s),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_scratch_memory_is_the_streams_own(allocations, name):
    side, call = Side(), calls()[name]
    call(side)
    call(None)
    assert allocations == [(4096, side), (4096, None)]


@pytest.mark.gpu
def test_attention_on_a_stream_beside_a_busy_one(dev):
    """The current stream still has to write a freed block of the workspace's size when the call goes to another one."""
    from test_gpu_kv_cache import gen, make_cache, make_table
    g = gen(1)
    lens = [3000, 50, 1200]
    table, pages, _ = make_table(g, dev, lens, 16, extra=400)
    c = make_cache(g, dev, pages, 2, 16, 64, "s8")
    qx = torch.randn((3, 8, 64), generator=g).to(dev)
    lengths = torch.tensor(lens, dtype=torch.int32, device=dev)
    want, out = torch.empty_like(qx), torch.empty_like(qx)
    q.paged_attention(c, table, lengths, qx, want)
    size = q.paged_attention_workspace_size(c, table, 8)
    work = torch.ones((4096, 4096), device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        block = torch.empty(size, dtype=torch.uint8, device=dev)
        for _ in range(4):
            torch.mm(work, work)
        block.fill_(0xFF)
        del block
        for _ in range(8):
            q.paged_attention(c, table, lengths, qx, out, stream=side)
        side.synchronize()
        assert torch.equal(out, want)
        torch.cuda.synchronize()
    q.sync_status()
