"""Products whose rows end inside an MMA, a scale tile or a stage (K any multiple of 32), by each kernel,
against 64 bits; bounds as in tests/test_gpu_act.py.

Scale bytes past the last block of x's rows may hold anything but NaN, and so may those of w's: they
meet elements that the copies leave zero."""
import numpy as np
import pytest
import torch

import act_reference as ref

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"


@pytest.fixture(params=[1, 2, 3, 4], ids=["narrow", "pairs", "pairs-2", "pairs-4"])
def forced(request):
    prev = w4.testing_set_act_kernel(request.param)
    yield request.param
    w4.testing_set_act_kernel(prev)


def _values(codes, tiles, form, K):
    s = ref.untile(tiles.cpu().numpy(), codes.shape[0], K // ref.BLOCK[form])
    return torch.from_numpy(ref.values(codes.cpu().numpy(), s, form)).to(DEV)


def _fill_past_blocks(tiles, rows, blocks, byte):
    """Bytes of the rows' scale words past their last block."""
    t = tiles.cpu().numpy().copy()
    r = np.arange(rows)[:, None]
    c = np.arange(blocks, t.shape[1] * 4)[None]
    t[r // 128, c // 4, r % 32 * 16 + r // 32 % 4 * 4 + c % 4] = byte
    return torch.from_numpy(t).to(DEV)


# K % 256 of 32, 64, 96, 128, 160, 192, 224 for 4-bit x; more than one tile a pair in the last but one
SHAPES = [(300, 264, 544), (257, 520, 1120), (130, 136, 96), (700, 1001, 2080), (300, 130, 1184),
          (129, 8, 32), (600, 264, 4288), (2100, 6144, 736), (50, 300, 8928)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
def test_rows_that_end_inside_a_stage(forced, form, M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    blocks = K // ref.BLOCK[form]
    x = torch.randn(M, K, device=DEV, generator=g) * torch.exp(
        torch.randn(M, 1, device=DEV, generator=g))
    xc, xs, rows = w4.act_quantize(x.bfloat16(), form)
    w = torch.randn(N, K, device=DEV, generator=g)
    wc, ws, wr = w4.act_quantize(w.bfloat16(), form)  # rows of weights in the same format
    xh, wh = _values(xc, xs, form, K), _values(wc, ws, form, K)
    S = torch.full((1,), 0.37, device=DEV)
    # the largest scale that is not NaN, the smallest and one between
    for byte in ((0x7E, 0x01, 0x38) if form == "nvfp4" else (0xFE, 0x00, 0x7F)):
        sx, sw = (_fill_past_blocks(t, n, blocks, byte) for t, n in ((xs, M), (ws, N)))
        y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
        if form == "nvfp4":
            w4.nvfp4_matmul_act(xc, sx, rows, wc, sw, S, y=y[:M])
            f = rows.double()[:, None] * S.double()
        else:
            w4.mxfp4_matmul_act(xc, sx, wc, sw, y=y[:M])
            f = 1.0
        want, terms = xh @ wh.T * f, xh.abs() @ wh.abs().T * f
        tol = 2.0 ** -8 * want.abs() + (K * 2.0 ** -27 + 2.0 ** -22) * terms
        off = (y[:M].double() - want).abs()
        assert (off <= tol).all(), f"byte {byte:#x}: {int((~(off <= tol)).sum())} of {off.numel()}"
        assert (y[M] == 7).all()
    assert w4.w4a16_device_status() == 0
