"""What sample refuses on the host, before anything is launched (no GPU
needed)."""
import ctypes

import pytest

from test_kv_abi import P, lib  # noqa: F401


def call(lib, logits=P, type=1, rows=3, vocabulary=100, stride=100, random=P, tokens=P):
    return lib.i8q_sample(logits, type, rows, vocabulary, stride, random, None, tokens, None, None)


@pytest.mark.parametrize("what,kw", [
    (b"type", dict(type=2)), (b"rows must", dict(rows=-1)), (b"rows must", dict(rows=(1 << 24) + 1)),
    (b"vocabulary must", dict(vocabulary=0)), (b"vocabulary must", dict(vocabulary=(1 << 20) + 1, stride=1 << 21)),
    (b"NULL", dict(logits=None)), (b"NULL", dict(random=None)), (b"NULL", dict(tokens=None)),
    (b"overlap", dict(stride=99)), (b"aligned", dict(logits=ctypes.c_void_p(4097))),
    (b"aligned", dict(logits=ctypes.c_void_p(4098), type=0)),
])
def test_refused(lib, what, kw):  # noqa: F811
    assert call(lib, **kw) == -1
    assert what in lib.i8q_last_error()


def test_no_rows(lib):  # noqa: F811
    assert call(lib, rows=0, logits=None) == 0


@pytest.mark.parametrize("which", ["random", "temperature", "top_k", "top_p", "min_p", "tokens", "logprobs"])
def test_rows_numbers_that_are_not_aligned(lib, which):  # noqa: F811
    """The kernel would read or write at an address that a GPU faults at."""
    from int8_quantized_gb300 import _lib
    at = {n: 4098 if n == which else 4096 for n in ("random", "tokens", "logprobs")}
    s = _lib.SamplingStruct(**{n: 4098 if n == which else 4096 for n in ("temperature", "top_k", "top_p", "min_p")})
    assert lib.i8q_sample(P, 1, 3, 100, 100, at["random"], ctypes.byref(s), at["tokens"], at["logprobs"], None) == -1
    assert b"aligned to their type" in lib.i8q_last_error()
