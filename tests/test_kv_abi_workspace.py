"""The size of paged_attention's workspace is 0, with the reason, for every
argument that the call itself refuses (no GPU needed)."""
import ctypes

import pytest

from test_kv_abi import attend, cache, lib, table  # noqa: F401

HUGE = dict(c=dict(kv_heads=60000, page_size=1 << 20, page_stride=1 << 50, head_stride=1 << 30),
            t=dict(max_pages=2000, stride=2000), q_heads=60000)


@pytest.mark.parametrize("what,code,kw", [
    (b"keeps scores", -1, dict(c=dict(score=None), accumulate=1)),
    (b"out of range", -2, HUGE),
    (b"out of range", -1, dict(t=dict(sequences=65536), q_heads=40000)),
    (b"multiple of kv_heads", -1, dict(q_heads=3)),
    (b"needs k_scale", -1, dict(c=dict(k_scale=None))),
    (b"overlap", -1, dict(t=dict(stride=1))),
])
def test_size_and_call_refuse_alike(lib, what, code, kw):  # noqa: F811
    c, t = cache(**kw.get("c", {})), table(**kw.get("t", {}))
    heads, accumulate = kw.get("q_heads", 4), kw.get("accumulate", 0)
    assert attend(lib, c=c, t=t, q_heads=heads, accumulate=accumulate) == code
    assert what in lib.i8q_last_error()
    assert lib.i8q_paged_attention_workspace_size(ctypes.byref(c), ctypes.byref(t), heads, accumulate) == 0
    assert what in lib.i8q_last_error() and b"workspace_size" in lib.i8q_last_error()


def test_size_without_scores_to_keep(lib):  # noqa: F811
    assert lib.i8q_paged_attention_workspace_size(ctypes.byref(cache(score=None)), ctypes.byref(table()), 4, 0) > 0
