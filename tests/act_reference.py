"""Quantized activations in plain numpy, 64 bits, for the tests (no GPU).

Written from the formats' description in include/w4a16.h, value by value; shares nothing with the
kernels."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# the non-negative finite E4M3 values, by code
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


def nearest(v, grid):
    """Codes (sign apart) of the values of `grid` nearest to |v|, ties to the even code."""
    a = np.minimum(np.abs(v), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def quantize(y, form):
    """float64 [M, K] -> (values of the elements, values of the scales [M, blocks], row scales)"""
    M, K = y.shape
    b = y.reshape(M, -1, BLOCK[form])
    top = np.abs(b).max(2)
    if form == "nvfp4":
        a = np.maximum(np.abs(y).max(1), 2.0 ** -80)
        s = E4M3[np.minimum(np.searchsorted(E4M3, 448 * top / a[:, None]), 126)]
        v = 2688 * b / np.where(s > 0, s * a[:, None], 1)[..., None]
        e = np.where(s[..., None] > 0, np.copysign(E2M1[nearest(v, E2M1)], b), 0)
        return e.reshape(M, K), s, a / 2688
    X = np.where(top > 0, np.frexp(top)[1] - 1 - (2 if form == "mxfp4" else 8), -127)
    s = 2.0 ** np.maximum(X, -127)
    grid = E2M1 if form == "mxfp4" else E4M3
    e = np.copysign(grid[nearest(b / s[..., None], grid)], b)
    return np.where(top[..., None] > 0, e, 0).reshape(M, K), s, None


def untile(t, R, C):
    """uint8 tiles [ceil(R/128), ceil(C/4), 512] -> scales [R, C]"""
    r, c = np.arange(R)[:, None], np.arange(C)[None, :]
    return t[r // 128, c // 4, r % 32 * 16 + r // 32 % 4 * 4 + c % 4]


def element_values(codes, form):
    if form == "mxfp8":
        mag = np.append(E4M3, np.nan)[codes & 127]
        return np.where(codes >> 7, -mag, mag)
    c = np.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1)
    return np.where(c >> 3, -E2M1[c & 7], E2M1[c & 7])


def scale_values(b, form):
    if form == "nvfp4":
        return np.append(E4M3, np.nan)[b & 127]
    return np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))


def values(codes, scales, form):
    """What codes and scales [R, blocks] stand for, without a row's or tensor's scale."""
    e = element_values(codes, form)
    s = scale_values(scales, form)
    return (e.reshape(e.shape[0], s.shape[1], -1) * s[..., None]).reshape(e.shape)


def rmsnorm(x, residual, weight, eps):
    """(h * weight, 1 / rms, h) of BF16 values as float64; h is rounded to BF16."""
    import torch

    h = x if residual is None else torch.from_numpy((x + residual).astype(np.float32)).bfloat16().double().numpy()
    return h * weight, 1 / np.sqrt((h * h).mean(1) + eps), h
