"""What the key/value cache entry points refuse, on the host and before
anything is launched (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from int8_quantized_gb300 import _lib, build
    build.build()
    return _lib.load()


P = ctypes.c_void_p(4096)


def cache(**kw):
    from int8_quantized_gb300 import _lib
    H, ps, D = kw.get("kv_heads", 2), kw.get("page_size", 16), kw.get("head_dim", 64)
    f = dict(k=4096, v=4096, k_scale=4096, v_scale=4096, score=4096, type=_lib.S8, pages=10, kv_heads=H, page_size=ps,
             head_dim=D, page_stride=H * ps * D, head_stride=ps * D, token_stride=D, scale_page_stride=H * ps,
             scale_head_stride=ps, scale_token_stride=1)
    if kw.get("type") == _lib.BF16:
        f.update(k_scale=None, v_scale=None)
    f.update(kw)
    return _lib.KVCacheStruct(**f)


def table(**kw):
    from int8_quantized_gb300 import _lib
    f = dict(table=4096, sequences=3, max_pages=4, stride=4)
    f.update(kw)
    return _lib.PageTableStruct(**f)


def rotary(**kw):
    from int8_quantized_gb300 import _lib
    f = dict(positions=4096, position_stride=8, axes=2, cos=4096, sin=4096, rows=100, pairs=32,
             pair_axis=bytes([0, 1] * 16), interleaved=0)
    f.update(kw)
    return _lib.RotaryStruct(**f)


def append(lib, c=None, t=None, seq=P, index=P, tokens=8, type=1, k=P, v=P, q=P, q_heads=4, q_out=P, rot=None):
    return lib.i8q_kv_append(ctypes.byref(c or cache()), ctypes.byref(t or table()), seq, index, tokens, type, k, 128,
                             64, v, 128, 64, q, 256, 64, q_heads, q_out, 256, 64,
                             None if rot is None else ctypes.byref(rot), None)


def gather(lib, c=None, t=None, seq=P, index=P, tokens=8, type=1, k=P, v=P):
    return lib.i8q_kv_gather(ctypes.byref(c or cache()), ctypes.byref(t or table()), seq, index, tokens, type, k, 128,
                             64, v, 128, 64, None)


def attend(lib, c=None, t=None, lengths=P, type=1, q=P, q_heads=4, out=P, scale=0.125, window=0, accumulate=0, ws=P,
           ws_bytes=1 << 40):
    return lib.i8q_paged_attention(ctypes.byref(c or cache()), ctypes.byref(t or table()), lengths, type, q, 256, 64,
                                   q_heads, out, 256, 64, None, scale, window, accumulate, ws, ws_bytes, None)


def evict(lib, c=None, t=None, n=None, lengths=P, kept=P, budget=32, sink=2, recent=4):
    return lib.i8q_kv_evict(ctypes.byref(c or cache()), ctypes.byref(t or table()), lengths,
                            ctypes.byref(n or table(max_pages=2, stride=2)), kept, budget, sink, recent, None, None)


CALLS = [append, gather, attend, evict]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("what,fields,code", [
    (b"type", dict(type=0), -1), (b"type", dict(type=3), -1), (b"NULL", dict(k=None), -1), (b"NULL", dict(v=None), -1),
    (b"needs k_scale", dict(k_scale=None), -1), (b"needs k_scale", dict(v_scale=None), -1),
    (b"no scales", dict(type=1, k_scale=4096), -1), (b"out of range", dict(pages=0), -1),
    (b"out of range", dict(pages=1 << 31), -1), (b"out of range", dict(kv_heads=0), -1),
    (b"out of range", dict(page_size=0), -1), (b"out of range", dict(page_size=-4), -1),
    (b"head_dim", dict(head_dim=0), -1), (b"multiple of 16", dict(head_dim=72, token_stride=80), -2),
    (b"multiple of 16", dict(head_dim=272), -2), (b"overlap", dict(token_stride=48), -1),
    (b"overlap", dict(page_stride=0), -1), (b"overlap", dict(head_stride=-1024), -1),
    (b"16 bytes", dict(token_stride=72), -1), (b"16 bytes", dict(page_stride=2056), -1),
    (b"16 bytes", dict(type=1, token_stride=68), -1), (b"scale strides", dict(scale_token_stride=0), -1),
    (b"aligned", dict(k=4104), -1), (b"aligned", dict(v=4097), -1),
])
def test_cache_refusals(lib, call, what, fields, code):
    assert call(lib, c=cache(**fields)) == code
    assert what in lib.i8q_last_error()


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("what,fields", [
    (b"NULL", dict(table=None)), (b"no rows", dict(sequences=0)), (b"too many", dict(sequences=1 << 20)),
    (b"no rows", dict(max_pages=0)), (b"2^31", dict(max_pages=1 << 27, stride=1 << 27)), (b"overlap", dict(stride=3)),
])
def test_table_refusals(lib, call, what, fields):
    assert call(lib, t=table(**fields)) == -1
    assert what in lib.i8q_last_error()


def test_null_structs(lib):
    assert lib.i8q_kv_gather(None, ctypes.byref(table()), P, P, 1, 1, P, 1, 1, P, 1, 1, None) == -1
    assert lib.i8q_kv_gather(ctypes.byref(cache()), None, P, P, 1, 1, P, 1, 1, P, 1, 1, None) == -1
    assert lib.i8q_paged_attention_workspace_size(None, ctypes.byref(table()), 4, 0) == 0


@pytest.mark.parametrize("what,kw", [
    (b"tokens", dict(tokens=-1)), (b"type", dict(type=2)), (b"NULL", dict(seq=None)), (b"NULL", dict(index=None)),
    (b"NULL", dict(k=None)), (b"NULL", dict(v=None)), (b"NULL", dict(q=None)), (b"NULL", dict(q_out=None)),
    (b"q_heads", dict(q_heads=-1)),
])
def test_append_refusals(lib, what, kw):
    assert append(lib, **kw) == -1
    assert what in lib.i8q_last_error()


@pytest.mark.parametrize("what,kw", [
    (b"pairs", dict(pairs=0)), (b"pairs", dict(pairs=33)), (b"axes", dict(axes=0)), (b"axes", dict(axes=5)),
    (b"NULL", dict(positions=None)), (b"NULL", dict(cos=None)), (b"NULL", dict(sin=None)), (b"rows", dict(rows=0)),
    (b"overlap", dict(position_stride=7)), (b"pair_axis", dict(pair_axis=bytes([0] * 31 + [2]))),
])
def test_rotary_refusals(lib, what, kw):
    assert append(lib, rot=rotary(**kw)) == -1
    assert what in lib.i8q_last_error()


@pytest.mark.parametrize("what,kw", [
    (b"tokens", dict(tokens=-1)), (b"type", dict(type=3)), (b"NULL", dict(seq=None)), (b"NULL", dict(k=None)),
    (b"NULL", dict(v=None)),
])
def test_gather_refusals(lib, what, kw):
    assert gather(lib, **kw) == -1
    assert what in lib.i8q_last_error()


def test_attention_refusals(lib):
    for what, kw in [(b"type", dict(type=2)), (b"NULL", dict(lengths=None)), (b"NULL", dict(q=None)),
                     (b"NULL", dict(out=None)), (b"multiple of kv_heads", dict(q_heads=3)),
                     (b"multiple of kv_heads", dict(q_heads=0)), (b"window", dict(window=-1)),
                     (b"NaN", dict(scale=float("nan"))), (b"keeps scores", dict(accumulate=1, c=cache(score=None))),
                     (b"workspace", dict(ws=None)), (b"workspace", dict(ws=ctypes.c_void_p(4096 + 16))),
                     (b"workspace", dict(ws_bytes=0))]:
        assert attend(lib, **kw) == -1, kw
        assert what in lib.i8q_last_error(), kw
    need = lib.i8q_paged_attention_workspace_size(ctypes.byref(cache()), ctypes.byref(table()), 4, 1)
    assert need > 0
    assert attend(lib, accumulate=1, ws_bytes=need - 1) == -1 and b"workspace" in lib.i8q_last_error()
    for heads in (0, 3, -2):
        assert lib.i8q_paged_attention_workspace_size(ctypes.byref(cache()), ctypes.byref(table()), heads, 0) == 0
        assert b"q_heads" in lib.i8q_last_error()


def test_evict_refusals(lib):
    for what, kw in [(b"no scores", dict(c=cache(score=None))), (b"NULL", dict(lengths=None)), (b"NULL", dict(kept=None)),
                     (b"differ in sequences", dict(n=table(sequences=2))), (b"budget", dict(budget=0)),
                     (b"budget", dict(budget=-3)), (b"budget", dict(budget=1 << 31)), (b"sink", dict(sink=-1)), (b"sink", dict(recent=-1)),
                     (b"sink", dict(sink=30)), (b"sink", dict(sink=33)), (b"NULL", dict(n=table(table=None)))]:
        assert evict(lib, **kw) == -1, kw
        assert what in lib.i8q_last_error(), kw


def test_binding_refuses_what_the_library_cannot_see():
    """Types, devices and shapes that only the tensors know (CPU tensors never reach the library)."""
    import torch

    import int8_quantized_gb300 as q
    k = torch.zeros((2, 2, 16, 64), dtype=torch.int8)
    s = torch.zeros((2, 2, 16))
    with pytest.raises(TypeError, match="CUDA"):
        q.KVCache(k, k, s, s)
    for bad in (k[0], "k", None):
        with pytest.raises(TypeError, match="CUDA"):
            q.KVCache(bad, bad, s, s)
    t = torch.zeros((1, 1), dtype=torch.int32)
    from int8_quantized_gb300 import _i32, _page_table, _rows
    with pytest.raises(TypeError, match="int32"):
        _page_table(t)
    with pytest.raises(TypeError, match="int32"):
        _i32(t, "seq", 1)
    with pytest.raises(TypeError, match="CUDA"):
        _rows(k, "q", (2, 2, 64), torch.int8)


def test_attention_refuses_lines_past_32_bits(lib):
    """A sequence whose row of the table times the heads cannot be cut by 32-bit positions."""
    huge = dict(c=cache(kv_heads=60000, page_size=1 << 20, page_stride=1 << 50, head_stride=1 << 30),
                t=table(max_pages=2000, stride=2000), q_heads=60000)
    assert attend(lib, **huge) == -2
    assert b"out of range" in lib.i8q_last_error()
