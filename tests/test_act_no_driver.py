"""Without a driver the activations' functions refuse their tensors as ever."""
import pytest
import torch


@pytest.mark.skipif(torch.cuda.is_available(), reason="a machine without a driver")
def test_tensors_without_a_driver(cuda_lib):
    import gemv_w4a16_group_gb300 as w4

    x, s = torch.zeros(2, 64).bfloat16(), torch.zeros(8, 4, dtype=torch.uint8)
    for call in (lambda: w4.act_quantize(x), lambda: w4.act_rmsnorm(x, x[0]),
                 lambda: w4.fp4_prepare_scales(s),
                 lambda: w4.mxfp4_matmul_act(s, s, s, s)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
