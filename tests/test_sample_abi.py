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
