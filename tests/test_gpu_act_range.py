"""Activations in 4 and 8 bits at the ends of fp32's range, against tests/act_reference.py (64 bits).

Behind the norm y = h * weight / rms is rounded to fp32 and then, where that falls on a border between
codes, moved to the side of the exact value; one that falls beside a border may have crossed it by what
fp32 does not hold of 1 / rms, 2^-24 of itself: MX codes and scales are those of some y (1 + d),
|d| <= 2^-23.
Codes and scales of BF16 rows are exact, and a product's bound is that of tests/test_gpu_act.py; a
result below BF16's normal range is off by half of its smallest step, 2^-134, more."""
import numpy as np
import pytest
import torch

import act_reference as ref

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"


def _f64(t):
    return t.detach().double().cpu().numpy()


def _held(codes, scales, form, K):
    b = ref.untile(scales.cpu().numpy(), codes.shape[0], K // ref.BLOCK[form])
    return ref.element_values(codes.cpu().numpy(), form), ref.scale_values(b, form)


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


# ---- NVFP4: blocks far below their row -----------------------------------------------------
def test_block_far_below_its_row():
    """448 max|block| / a below fp32's range: the block's scale is still E4M3's smallest."""
    K = 128
    x = torch.zeros(3, K)
    x[:, 0] = torch.tensor([3.3e38, -2.0 ** 127, 2.0 ** 100])
    x[0, 16:32] = 2.0 ** -133
    x[1, 32:48] = -(2.0 ** -126)
    x[2, 48:64] = 2.0 ** -120
    x[:, 127] = 2.0 ** -60
    x = x.bfloat16()
    codes, scales, rows = w4.act_quantize(x.to(DEV), "nvfp4")
    e, s = _held(codes, scales, "nvfp4", K)
    we, ws, wr = ref.quantize(_f64(x), "nvfp4")
    assert ws[0, 1] == ws[1, 2] == ws[2, 3] == 2.0 ** -9
    assert np.array_equal(s, ws) and np.array_equal(e, we)
    assert (np.abs(_f64(rows) - wr) <= 2.0 ** -23 * wr).all()


# ---- NVFP4 products: a row's scale times the tensor's --------------------------------------
@pytest.mark.parametrize("kernel,M,K", [(1, 5, 256), (1, 5, 4096), (1, 40, 4096), (1, 3, 1024),
                                        (2, 140, 256), (3, 140, 1024), (4, 140, 2048)])
@pytest.mark.parametrize("N", [130, 136])
def test_scales_whose_product_leaves_fp32(kernel, M, N, K):
    """Rows of 2^-78 to 2^120 by tensors of 2^-80 to 2^60: r S may leave fp32's range where y
    does not, and rows of zeros stay zeros."""
    g = torch.Generator().manual_seed(K)
    size = torch.tensor([-78.0, -60, -20, 0, 40, 80, 120]).repeat(20)[:M]
    x = (torch.randn(M, K, generator=g) * torch.exp2(size)[:, None]).bfloat16()
    x[M - 1] = 0
    q = w4.act_quantize(x.to(DEV), "nvfp4")
    codes, scales, _ = w4.nvfp4_quantize(torch.randn(N, K, generator=g).to(DEV))
    codes[3] = 0
    tiles = w4.fp4_prepare_scales(scales)
    e, s = _held(q[0], q[1], "nvfp4", K)
    xh = (e.reshape(M, -1, 16) * s[..., None]).reshape(M, K)
    wh = ref.values(codes.cpu().numpy(), scales.cpu().numpy(), "nvfp4")
    sums, terms = xh @ wh.T, np.abs(xh) @ np.abs(wh).T
    prev = w4.testing_set_act_kernel(kernel)
    try:
        for power in (-80, -60, -30, 0, 30, 60):
            S = torch.tensor([1.37 * 2.0 ** power], device=DEV)
            y = _f64(w4.nvfp4_matmul_act(q[0], q[1], q[2], codes, tiles, S))
            f = _f64(q[2])[:, None] * _f64(S)
            want, bound = sums * f, terms * f
            tol = 2.0 ** -8 * np.abs(want) + (K * 2.0 ** -27 + 2.0 ** -22) * bound + 2.0 ** -134
            top = float(torch.finfo(torch.bfloat16).max)
            big = np.abs(want) - tol > top  # infinite for certain; else near it, or in range
            near = (np.abs(want) + tol > top) & ~big
            assert (y[big] == np.copysign(np.inf, want[big])).all()
            inside = ~big & ~near
            off = np.abs(y[inside] - want[inside])
            assert (off <= tol[inside]).all(), f"2^{power}: {(~(off <= tol[inside])).sum()}"
            assert (y[:, 3] == 0).all() and (y[M - 1] == 0).all()
    finally:
        w4.testing_set_act_kernel(prev)
    assert w4.w4a16_device_status() == 0


# ---- the norm: products that leave fp32 ----------------------------------------------------
@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("M,K", [(5, 64), (9, 1056), (400, 4096)])
def test_norm_of_products_below_fp32(form, M, K):
    """Rows of 2^-74 by weights of 2^-70 to 1: h * weight leaves fp32's normal range, and fp32's
    range, where h * weight / rms does not."""
    eps = float(np.float32(1e-30))
    h = (_randn(M, K, seed=K) * torch.exp2(torch.linspace(-78, -60, M))[:, None]).bfloat16()
    block = torch.arange(K) // 32
    weight = (_randn(K, seed=K + 1) * torch.exp2(-(block % 8) * 10.0)).bfloat16()
    h[1, 64:] = 0
    codes, scales, _, _ = w4.act_rmsnorm(h.to(DEV), weight.to(DEV), form, eps=eps)
    e, s = _held(codes, scales, form, K)
    z, rinv, _ = ref.rmsnorm(_f64(h), None, _f64(weight), eps)
    fits = False
    for d in (-2.0 ** -23, 0, 2.0 ** -23):
        we, ws, _ = ref.quantize(z * rinv[:, None] * (1 + d), form)
        fits |= (e == we) & (np.repeat(s == ws, 32, 1))
    assert fits.all(), f"{(~fits).sum()} of {fits.size}"


@pytest.mark.parametrize("form", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("power", [60, 50])
def test_norm_of_products_above_fp32(form, power):
    """Rows of 2^50 by weights of 2^80: h * weight is past fp32's range, h * weight / rms is not.
    At 2^60 the sum of the row's squares is, too (512 * 2^120), and the row is NaN."""
    M, K = 6, 512
    h = (_randn(M, K, seed=1) * 2.0 ** power).bfloat16()
    h[2, :64] *= 2.0 ** -80
    weight = (_randn(K, seed=2) * torch.exp2((torch.arange(K) // 32 % 3) * 40.0)).bfloat16()
    codes, scales, _, _ = w4.act_rmsnorm(h.to(DEV), weight.to(DEV), form)
    e, s = _held(codes, scales, form, K)
    if power == 60:
        assert ((_f64(h) ** 2).sum(1) > 2.0 ** 128).all() and np.isnan(s).all()
        return
    z, rinv, _ = ref.rmsnorm(_f64(h), None, _f64(weight), 1e-6)
    assert np.abs(z).max() > 2.0 ** 128
    fits = False
    for d in (-2.0 ** -23, 0, 2.0 ** -23):
        we, ws, _ = ref.quantize(z * rinv[:, None] * (1 + d), form)
        fits |= (e == we) & (np.repeat(s == ws, 32, 1))
    assert fits.all(), f"{(~fits).sum()} of {fits.size}"


# ---- scale tiles of as many rows as an int counts ------------------------------------------
def test_scale_tiles_of_the_most_rows():
    R = (1 << 31) - 1
    scales = torch.arange(1 << 20, device=DEV).mul_(2654435761).bitwise_right_shift_(7).to(torch.uint8)
    scales = scales.repeat(1 << 11)[:R].view(R, 1)
    tiles = w4.fp4_prepare_scales(scales)
    assert tiles.shape == (1 << 24, 1, 512)
    for first in (0, 12345, (1 << 24) - 100):  # blocks of 128 rows
        part = tiles[first:first + 100]
        full = ref.untile(part.cpu().numpy(), 12800, 4)
        want = np.zeros((12800, 4), np.uint8)
        rows = scales[first * 128:first * 128 + 12800].cpu().numpy()
        want[:rows.shape[0], :1] = rows
        assert np.array_equal(full, want)
