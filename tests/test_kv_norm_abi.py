"""What kv_append refuses about norms, on the host and before anything is
launched (no GPU needed)."""
import ctypes

import pytest

from test_kv_abi import P, cache, lib, rotary, table  # noqa: F401


def call(lib, norm, q_heads=4, rot=None, type=1):
    qp = P if q_heads else None
    return lib.i8q_kv_append_norm(ctypes.byref(cache()), ctypes.byref(table()), P, P, 8, type, P, 128, 64, P, 128, 64, qp,
                                  256, 64, q_heads, qp, 256, 64, rot, ctypes.byref(norm), None)


@pytest.mark.parametrize("what,fields,heads", [
    (b"type", dict(type=2), 4), (b"type", dict(type=-1), 4), (b"eps", dict(eps=-1.0), 4),
    (b"eps", dict(eps=float("nan")), 4), (b"eps", dict(eps=float("inf")), 4), (b"needs q", {}, 0),
    (b"aligned", dict(q_weight=4098), 4), (b"aligned", dict(k_weight=4097, type=1), 4),
])
def test_refused(lib, what, fields, heads):  # noqa: F811
    from int8_quantized_gb300 import _lib
    f = dict(q_weight=4096, k_weight=4096, type=0, eps=1e-6)
    f.update(fields)
    assert call(lib, _lib.HeadNormStruct(**f), heads) == -1
    assert what in lib.i8q_last_error()


def test_the_other_arguments_are_refused_as_without_norms(lib):  # noqa: F811
    from int8_quantized_gb300 import _lib
    n = _lib.HeadNormStruct(4096, 4096, 0, 1e-6)
    assert call(lib, n, type=2) == -1
    assert call(lib, n, rot=ctypes.byref(rotary(pairs=40))) == -1
    assert b"pairs" in lib.i8q_last_error()
