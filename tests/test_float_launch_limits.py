"""Sizes whose grids the runtime cannot take (2^32 threads along a dimension)
are refused as SHAPE before anything is enqueued (no GPU needed: none of these
calls reaches one)."""
import ctypes

from integer_only_nn_amd import _lib

lib = _lib.lib()
SHAPE = 2
A = ctypes.c_void_p(0x1000)  # never dereferenced


def test_linear_fwd():
    f = lambda B, IN, OUT: lib.dfp8_linear_fwd(A, A, A, A, None, 0, None, None, A, 1, B, IN, OUT, None, A, 1 << 40, None)  # noqa: E731
    assert f(1, 16, 1 << 30) == SHAPE and f(1, 5, 1 << 30) == SHAPE and f(1, 0, 1 << 30) == SHAPE
    assert f(1 << 30, 16, 64) == SHAPE and f(1 << 17, 100, 1 << 19) == SHAPE
    assert b"tiles" in lib.ionn_last_error()


def test_linear_bwd():
    def f(B, IN, OUT, dX=A, G=A):
        return lib.dfp8_linear_bwd(A, A, 1, 1, A, A, A, A, A, A, dX, G, None, B, IN, OUT, None, A, 1 << 40, None)
    assert f(1, 1 << 30, 8) == SHAPE and f(1, 1 << 30, 8, G=None) == SHAPE and f(1, 1 << 30, 8, dX=None) == SHAPE
    assert f(64, 1 << 29, 64) == SHAPE  # (either gradient alone would be taken)
    assert f(1 << 30, 64, 64, G=None) == SHAPE
    assert b"tiles" in lib.ionn_last_error()


def test_adamw():
    arr = (ctypes.c_void_p * 1)(0x1000)

    def f(n, bits):
        return lib.ionn_adamw_step(1, arr, arr, 1, arr, arr, arr, bits, (ctypes.c_int64 * 1)(n), 1, 1e-3, 0.9, 0.999, 1e-8,
                                   0.0, None, None, None, None, None)
    assert f(1 << 35, 8) == SHAPE and f(1 << 36, 32) == SHAPE
