"""What the MatMulNBits entry points refuse, on the host and before anything
is launched, and the packed size (no GPU needed)."""
import ctypes

import pytest

from test_kv_abi import P, lib  # noqa: F401

F32, BF16 = 0, 1
ODD = ctypes.c_void_p(4097)


def pack(lib, N=32, K=64, block=32, B=P, scales=P, stype=BF16, zero=P, packed=P, size=1 << 40):
    return lib.i8q_matmul_nbits_pack(N, K, block, B, scales, stype, zero, packed, size, None)


def product(lib, A=P, type=BF16, M=3, lda=64, packed=P, size=1 << 40, N=32, K=64, block=32, stype=BF16, zero=1, bias=None,
            Y=P, ldy=32):
    return lib.i8q_matmul_nbits(A, type, M, lda, packed, size, N, K, block, stype, zero, bias, Y, ldy, None)


@pytest.mark.parametrize("call", [pack, product])
@pytest.mark.parametrize("what,kw,code", [
    (b"N and K", dict(N=0), -1), (b"N and K", dict(K=0), -1), (b"N and K", dict(N=-5), -1),
    (b"N and K", dict(K=1 << 31), -1), (b"scales must", dict(stype=2), -1), (b"block_size", dict(block=8), -2),
    (b"block_size", dict(block=0), -2), (b"block_size", dict(block=48), -2), (b"block_size", dict(block=512), -2),
    (b"NULL", dict(packed=None), -1), (b"aligned", dict(packed=ctypes.c_void_p(4104)), -1), (b"smaller", dict(size=100), -1),
])
def test_both_refuse(lib, call, what, kw, code):  # noqa: F811
    assert call(lib, **kw) == code
    assert what in lib.i8q_last_error()


@pytest.mark.parametrize("what,kw", [(b"NULL", dict(B=None)), (b"NULL", dict(scales=None)), (b"aligned", dict(scales=ODD)),
                                     (b"aligned", dict(scales=ctypes.c_void_p(4098), stype=F32))])
def test_pack_refuses(lib, what, kw):  # noqa: F811
    assert pack(lib, **kw) == -1
    assert what in lib.i8q_last_error()


@pytest.mark.parametrize("what,kw", [
    (b"type", dict(type=2)), (b"M must", dict(M=-1)), (b"M must", dict(M=1 << 31)), (b"NULL", dict(A=None)),
    (b"NULL", dict(Y=None)), (b"overlap", dict(lda=63)), (b"overlap", dict(ldy=31)), (b"aligned", dict(A=ODD)),
    (b"aligned", dict(Y=ODD)), (b"aligned", dict(bias=ctypes.c_void_p(4098))),
    (b"aligned", dict(A=ctypes.c_void_p(4098), type=F32)),
])
def test_product_refuses(lib, what, kw):  # noqa: F811
    assert product(lib, **kw) == -1
    assert what in lib.i8q_last_error()


def test_no_rows_is_nothing_to_do(lib):  # noqa: F811
    assert product(lib, M=0, A=None, Y=None) == 0


def test_packed_size(lib):  # noqa: F811
    size = lib.i8q_matmul_nbits_packed_size
    # tiles of 16 x 128: 1024 bytes of codes, 16 x 128 / block scales and zero points
    assert size(16, 128, 128, BF16, 0) == 1024 + 32
    assert size(17, 129, 32, F32, 1) == 4 * (1024 + 64 * 5)
    assert size(16, 200, 256, BF16, 1) == 2 * (1024 + 16 * 3)
    assert size(1 << 20, 1 << 16, 16, BF16, 0) == (1 << 16) * 512 * (1024 + 256)
    assert size(16, 128, 33, BF16, 0) == 0 and size(0, 128, 32, BF16, 0) == 0 and size(16, 128, 32, 3, 0) == 0
