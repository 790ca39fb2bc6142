"""Tensors of another device than the current one are refused before a launch: the kernels of the 4-
and 8-bit activations run on the current device, which may not reach another one's memory. (With one
GPU the current device's number is made to differ.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"


def _calls():
    M, N, K = 3, 16, 256
    x, weight = torch.randn(M, K, device=DEV).bfloat16(), torch.ones(K, device=DEV).bfloat16()
    w = torch.randn(N, K, device=DEV)
    c4, s4, S = w4.nvfp4_quantize(w)
    cm, sm = w4.mxfp4_quantize(w)
    t4, tm = w4.fp4_prepare_scales(s4), w4.fp4_prepare_scales(sm)
    q4, qm = w4.act_quantize(x), w4.act_quantize(x, "mxfp8")
    return {"scales": lambda: w4.fp4_prepare_scales(s4),
            "x": lambda: w4.act_quantize(x, "mxfp4"),
            "x ": lambda: w4.act_rmsnorm(x, weight),
            "x_codes": lambda: w4.nvfp4_matmul_act(*q4, c4, t4, S),
            "x_codes ": lambda: w4.mxfp4_matmul_act(qm[0], qm[1], cm, tm)}


def test_tensors_of_another_device(monkeypatch):
    calls = _calls()
    before = [call() for call in calls.values()]
    torch.cuda.synchronize()
    monkeypatch.setattr(w4, "_device", lambda: 1)
    for name, call in calls.items():
        with pytest.raises(ValueError, match=f"{name.strip()} must be on the current device, cuda:1"):
            call()
    monkeypatch.undo()
    assert len(before) == 5
    assert w4.w4a16_device_status() == 0


def test_each_tensor_is_looked_at(monkeypatch):
    """A tensor of its own on another device, among others that are on the current one."""
    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1

    M, N, K = 3, 16, 256
    x, weight = torch.randn(M, K, device=DEV).bfloat16(), torch.ones(K, device=DEV).bfloat16()
    w = torch.randn(N, K, device=DEV)
    c4, s4, S = w4.nvfp4_quantize(w)
    t4, q = w4.fp4_prepare_scales(s4), w4.act_quantize(x)
    y, out = torch.empty(M, N, device=DEV).bfloat16(), torch.empty_like(x)
    norm = dict(x=x, weight=weight, residual=x, residual_out=out, codes=q[0], scales=q[1],
                row_scales=q[2])
    product = dict(x_codes=q[0], x_scales=q[1], x_row_scales=q[2], codes=c4, scale_tiles=t4,
                   tensor_scale=S, y=y)
    for call, args in ((w4.act_rmsnorm, norm), (w4.nvfp4_matmul_act, product),
                       (w4.fp4_prepare_scales, dict(scales=s4, tiles=t4))):
        for name, t in args.items():
            with pytest.raises(ValueError, match=f"{name} must be on the current device"):
                call(**{**args, name: t.as_subclass(Elsewhere)})
    torch.cuda.synchronize()
    assert w4.w4a16_device_status() == 0
