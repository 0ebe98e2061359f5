"""The carried optimiser step's host-side checks (no GPU needed: none of these
calls reaches one)."""
import ctypes

from integer_only_nn_amd import _lib

lib = _lib.lib()
OK, ARG, SHAPE, RANGE, ALIGN = range(5)


def test_adamw_carried():
    arr = lambda *ps: (ctypes.c_void_p * len(ps))(*ps)  # noqa: E731
    num = lambda *ns: (ctypes.c_int64 * len(ns))(*ns)  # noqa: E731
    T = arr(0x1000, 0x2000)  # never dereferenced

    def f(L=2, p=T, g=T, gd=0, m=T, v=T, s=T, r=T, n=num(8, 300), t=1, lr=1e-3, b2=0.99, step=None):
        return lib.ionn_adamw_step_carried(L, p, g, gd, m, v, s, r, n, t, lr, 0.9, b2, 1e-8, 0.0, step, None, None, None, None)
    assert f(r=None) == ARG and f(r=arr(0x1000, None)) == ARG and f(s=None) == ARG and f(s=arr(None, 0x1000)) == ARG
    assert b"ionn_adamw_step_carried: tensor 0" in lib.ionn_last_error()
    assert f(L=0) == SHAPE and f(n=num(8, 0)) == SHAPE and f(gd=3) == ARG and f(p=arr(0x1000, 0x2002)) == ALIGN
    assert f(t=0) == RANGE and f(b2=1.0) == RANGE and f(step=ctypes.c_void_p(0x1001)) == ALIGN
