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
