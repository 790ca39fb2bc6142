"""The residual's sum in one array with its inputs: whole rows in place, or beside them; anything
between is refused before a launch."""
import pytest
import torch

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"


def test_sums_in_one_array_with_their_inputs():
    M, K = 37, 256
    weight = torch.ones(K, device=DEV).bfloat16()
    wide = torch.randn(M + 1, 3 * K, device=DEV).bfloat16()
    x, res, out = wide[:M, :K], wide[:M, K:2 * K], wide[:M, 2 * K:]

    def norm(x, res, out=None):
        # (places of rows past M are not written: they hold the same in every call)
        tiles = torch.zeros(1, K // 64, 512, dtype=torch.uint8, device=DEV)
        return w4.act_rmsnorm(x, weight, residual=res, residual_out=out, scales=tiles)

    want = norm(x.clone(), res.clone())
    got = norm(x, res, out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for other in (wide[1:, :K], wide[:M, K // 2:K // 2 + K], wide[1:, K:2 * K],
                  wide.view(-1)[:M * K].view(M, K)):
        before = wide.clone()
        with pytest.raises(w4.W4A16Error, match="INVALID"):
            norm(x, res, other)
        torch.cuda.synchronize()
        assert torch.equal(wide.view(torch.int16), before.view(torch.int16))
    got = norm(x, res, res)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert w4.w4a16_device_status() == 0
