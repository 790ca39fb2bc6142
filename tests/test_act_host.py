"""Activations in 4 and 8 bits without a GPU: sizes, refusals before any launch, and the
reference's own pins."""
import ctypes

import numpy as np
import pytest

import act_reference as ref

OK, INVALID, UNSUPPORTED, MISALIGNED = range(4)
A, B = 0x10000, 0x20000  # never dereferenced
NV, MX4, MX8 = range(3)


@pytest.fixture(scope="module")
def lib(cuda_lib):
    lib = ctypes.CDLL(cuda_lib)
    P, I, L, S, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                     ctypes.c_float)
    lib.fp4_scale_tiles_bytes.argtypes = [I, I]
    lib.fp4_scale_tiles_bytes.restype = S
    lib.fp4_prepare_scales.argtypes = [P, I, I, P, P]
    lib.act_quantize.argtypes = [P, L, I, I, I, P, P, P, P]
    lib.act_rmsnorm.argtypes = [P, L, P, L, P, L, P, F, I, I, I, P, P, P, P]
    lib.nvfp4_matmul_act.argtypes = [P, P, P, P, P, P, P, I, I, I, P]
    lib.mxfp4_matmul_act.argtypes = [P, P, I, P, P, P, I, I, I, P]
    return lib


def _quantize(lib, x=A, xs=256, M=3, K=256, form=NV, codes=A, scales=A, rows=A):
    return lib.act_quantize(x, xs, M, K, form, codes, scales, rows, None)


def _rmsnorm(lib, x=A, xs=256, res=None, rs=0, out=None, os_=0, w=A, eps=1e-6, M=3, K=256,
             form=NV, codes=A, scales=A, rows=A):
    return lib.act_rmsnorm(x, xs, res, rs, out, os_, w, eps, M, K, form, codes, scales, rows, None)


def _nv(lib, xc=A, xs=A, xr=A, c=A, s=A, S=A, y=B, M=3, N=8, K=256):
    return lib.nvfp4_matmul_act(xc, xs, xr, c, s, S, y, M, N, K, None)


def _mx(lib, xc=A, xs=A, form=MX4, c=A, s=A, y=B, M=3, N=8, K=256):
    return lib.mxfp4_matmul_act(xc, xs, form, c, s, y, M, N, K, None)


def test_tile_sizes(lib):
    nb = lib.fp4_scale_tiles_bytes
    assert nb(1, 1) == 512 and nb(128, 4) == 512 and nb(129, 5) == 2048
    assert nb(14336, 256) == 14336 * 256
    assert nb(0, 4) == nb(4, 0) == nb(-1, 4) == 0
    assert nb(1 << 30, 1 << 20) == (1 << 50)


def test_prepare_refusals(lib):
    f = lib.fp4_prepare_scales
    for args in [(None, 8, 4, A), (A, 8, 4, None), (A, 0, 4, A), (A, 8, 0, A), (A, -1, 4, A)]:
        assert f(*args, None) == INVALID
    assert f(A, 8, 4, A + 8, None) == MISALIGNED


@pytest.mark.parametrize("call", [_quantize, _rmsnorm])
def test_quantizer_refusals(lib, call):
    for k in ("x", "codes", "scales"):
        assert call(lib, **{k: None}) == INVALID
        assert call(lib, **{k: A + 8}) == MISALIGNED
    assert call(lib, rows=None) == INVALID
    assert call(lib, rows=A + 2) == MISALIGNED
    for k, v in [("M", 0), ("M", -1), ("K", 0), ("K", 16), ("K", 40), ("form", -1), ("form", 3),
                 ("xs", 248), ("xs", 260), ("xs", 0)]:
        assert call(lib, **{k: v}) == INVALID, (k, v)
    assert call(lib, K=65536 + 32, xs=1 << 20) == UNSUPPORTED


def test_rmsnorm_refusals(lib):
    assert _rmsnorm(lib, w=None) == INVALID
    assert _rmsnorm(lib, w=A + 2) == MISALIGNED
    for eps in (0.0, -1e-6, 1e-31, float("nan"), float("inf")):
        assert _rmsnorm(lib, eps=eps) == INVALID
    both = dict(res=A, rs=256, out=B, os_=256)
    assert _rmsnorm(lib, res=A, rs=256) == INVALID
    assert _rmsnorm(lib, out=A, os_=256) == INVALID
    for k in ("rs", "os_"):
        assert _rmsnorm(lib, **{**both, k: 128}) == INVALID
        assert _rmsnorm(lib, **{**both, k: 257}) == INVALID
    for k in ("res", "out"):
        assert _rmsnorm(lib, **{**both, k: A + 8}) == MISALIGNED


def test_product_refusals(lib):
    for k in ("xc", "xs", "xr", "c", "s", "S", "y"):
        assert _nv(lib, **{k: None}) == INVALID
        assert _nv(lib, **{k: A + 2}) == MISALIGNED
    for k in ("xc", "xs", "c", "s", "y"):
        for form in (MX4, MX8):
            assert _mx(lib, **{k: None, "form": form}) == INVALID
            assert _mx(lib, **{k: A + 8, "form": form}) == MISALIGNED
    assert _mx(lib, c=A + 16, form=MX8) == MISALIGNED
    for k in ("M", "N", "K"):
        for v in (0, -32):
            assert _nv(lib, **{k: v}) == INVALID and _mx(lib, **{k: v}) == INVALID
        big = {k: (1 << 23) + 128}
        assert _nv(lib, **big) == UNSUPPORTED and _mx(lib, **big) == UNSUPPORTED
    assert _nv(lib, K=48) == _mx(lib, K=48) == INVALID
    assert _mx(lib, K=160, form=MX8) == INVALID
    for form in (-1, NV, 3):
        assert _mx(lib, form=form) == INVALID


# ---- the reference's own pins ------------------------------------------------------------
def test_grids():
    assert ref.E4M3[[1, 7, 8, 56, 126]].tolist() == [2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1, 448]
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7, 0.2500001, 2.4999])
    assert ref.E2M1[ref.nearest(v, ref.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 0.5, 2]
    assert ref.E4M3[ref.nearest(np.array([17, 19, 464, 1e9, 2.0 ** -10, 3 * 2.0 ** -10]),
                                ref.E4M3)].tolist() == [16, 20, 448, 448, 0, 2.0 ** -8]


def test_quantize_pins():
    y = np.zeros((1, 32))
    y[0, :4] = [3, -0.75, 0.5, 0.2]
    e, s, _ = ref.quantize(y, "mxfp4")           # floor(log2 3) - 2 = -1
    assert s[0, 0] == 0.5 and e[0, :4].tolist() == [6, -1.5, 1, 0.5]
    e, s, _ = ref.quantize(y, "mxfp8")           # 1 - 8
    assert s[0, 0] == 2.0 ** -7 and e[0, :4].tolist() == [384, -96, 64, 26]
    e, s, r = ref.quantize(y, "nvfp4")
    assert r[0] == 3 / 2688 and s[0].tolist() == [448, 0] and e[0, :4].tolist() == [6, -1.5, 1, 0.5]
    e, s, r = ref.quantize(0 * y, "nvfp4")
    assert r[0] == 2.0 ** -80 / 2688 and not e.any() and not s.any()


def test_tiles_and_codes():
    t = np.zeros((2, 3, 512), np.uint8)
    t[1, 2, (37 % 32) * 16 + 1 * 4 + 3] = 9
    assert ref.untile(t, 200, 12)[128 + 37, 11] == 9
    assert ref.element_values(np.array([[0x2F]], np.uint8), "mxfp4").tolist() == [[-6, 1]]
    assert ref.element_values(np.array([[0xB8, 0x7E]], np.uint8), "mxfp8").tolist() == [[-1, 448]]
    assert ref.scale_values(np.array([127, 0, 130], np.uint8), "mxfp4").tolist() == [1, 2.0 ** -127, 8]
