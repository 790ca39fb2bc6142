"""Activations in 4 and 8 bits at the ends of fp32's range, against tests/act_reference.py (64 bits).

Codes and scales of BF16 rows are exact, as in tests/test_gpu_act.py."""
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
