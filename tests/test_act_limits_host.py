"""Refusals of the norm without a GPU. Every call here also has a misaligned weight, which is refused
after the rest: no call reaches a launch, on a machine with a GPU either."""
import ctypes

import pytest

INVALID, MISALIGNED = 1, 3
A = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib(cuda_lib):
    lib = ctypes.CDLL(cuda_lib)
    P, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.act_rmsnorm.argtypes = [P, L, P, L, P, L, P, F, I, I, I, P, P, P, P]
    return lib


def _rmsnorm(lib, x=A, xs=256, res=None, rs=0, out=None, os_=0, eps=1e-6, M=3, K=256):
    return lib.act_rmsnorm(x, xs, res, rs, out, os_, (1 << 30) + 2, eps, M, K, 0, 1 << 31, 1 << 32,
                           1 << 33, None)


def test_eps_that_leaves_fp32(lib):
    for eps in (1.1e30, 1e33, 3e38):
        assert _rmsnorm(lib, eps=eps) == INVALID
    for eps in (1e-30, 1.0, 1e30):
        assert _rmsnorm(lib, eps=eps) == MISALIGNED


def test_residual_out_that_overlaps_in_part(lib):
    """The sum may replace x or the residual as a whole, or lie beside them, in one array too."""
    B, row = 1 << 20, 2 * 256  # bytes of a row
    for name, stride in (("x", "xs"), ("res", "rs")):
        other = {"x": B, "xs": 256} if name == "res" else {"res": B, "rs": 256}

        def call(at, s, out, os_, **kw):
            return _rmsnorm(lib, **other, **{name: at, stride: s}, out=out, os_=os_, **kw)

        for at, s, out, os_ in [
                (A, 256, A + 16, 256),            # a few values further
                (A, 256, A + row, 256),           # a row further
                (A + row, 256, A, 256),
                (A, 512, A + row // 2, 512),      # half of a row, in rows of a wider array
                (A, 512, A + 3 * row // 2, 512),
                (A, 256, A, 512),                 # the same place in other steps
                (A, 512, A, 256),
                (A, 264, A + row, 320)]:
            assert call(at, s, out, os_) == INVALID, (name, at, s, out, os_)
        for at, s, out, os_ in [
                (A, 256, A, 256), (A, 512, A, 512),
                (A, 512, A + row, 512),           # the other half of the same rows
                (A + row, 512, A, 512),
                (A, 256, A + 3 * row, 256), (A + 3 * row, 256, A, 256),
                (A, 264, A + 3 * 528, 320)]:
            assert call(at, s, out, os_) == MISALIGNED, (name, at, s, out, os_)
        assert call(A, 256, A, 512, M=1) == MISALIGNED  # one row has no steps
        assert call(A, 256, A + 16, 512, M=1) == INVALID
