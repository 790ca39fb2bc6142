"""MX codes behind the norm against the exact row's, over tens of millions of values.

Bounds, before any run. 1 / rms is carried in two floats: with up to two pieces a thread (K up to 16384) a
thread sums 16 squares in each of two sums, and what an addition loses is known exactly; what is lost
of the sum of the losses is 16 of 2^-24 of 16 of 2^-24 of the sum, 2^-40; ten joins, as much again; the
root halves both; a guess within 2^-21.4 and one step of Newton leave 1.5 2^-42.8, the step's own
roundings 2^-43: 2^-39 in all. y = h * weight / rms is rounded to fp32 and then, where that falls on a
border between codes, moved to the side of the exact value. One that falls beside a border may have
crossed it by what fp32 does not hold of 1 / rms, 2^-24 of itself, so a code that is not the exact row's
lies within 2^-23 of a border, and about one in 10^8 does. Of 5 * 10^7 values 0.5 are expected, and more
than 4 have a chance of 2 in 10^4; with sums, root and product in plain fp32 about one in two million
is another, so that this test tells the two apart (it counts them, too)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"
EPS = 1e-6
GRID4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _elements(v, form):
    """Nearest values of the format, ties to the even code, of float64 v."""
    a = v.abs()
    if form == "mxfp8":
        step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
        step = torch.where(a >= 16 * step, 2 * step, step)
        step = torch.where((a < 8 * step) & (step > 2.0 ** -9), step / 2, step)
        return torch.copysign((torch.round(a / step) * step).clamp_max(448.0), v)
    grid = torch.tensor(GRID4, dtype=torch.float64, device=DEV)
    mid = (grid[1:] + grid[:-1]) / 2
    up, down = torch.bucketize(a, mid, right=True), torch.bucketize(a, mid)
    i = torch.where((up != down) & (up % 2 == 1), down, up)  # a tie: the even code
    return torch.copysign(grid[i], v)


def _exact(y, form):
    """(elements, scales) of float64 rows y [M, K]"""
    b = y.view(y.shape[0], -1, 32)
    X = torch.frexp(b.abs().amax(2))[1] - 1 - (2 if form == "mxfp4" else 8)
    s = torch.exp2(X.double())
    return _elements(b / s[..., None], form).view(y.shape), s


def _held(codes, tiles, form):
    M = codes.shape[0]
    if form == "mxfp8":
        e = codes.view(torch.float8_e4m3fn).double()
    else:
        c = torch.stack([codes & 15, codes >> 4], 2).view(M, -1).long()
        e = torch.tensor(GRID4, dtype=torch.float64, device=DEV)[c & 7] * (1 - 2 * (c >> 3))
    K = e.shape[1]
    rb, cb, _ = tiles.shape
    s = tiles.view(rb, cb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cb * 4)
    return e, torch.exp2(s[:M, :K // 32].double() - 127)


@pytest.mark.parametrize("form,K", [("mxfp8", 4096), ("mxfp4", 4096), ("mxfp8", 14336)])
def test_codes_behind_the_norm(form, K):
    M, turns = 2048, (50 * 10 ** 6 + 2048 * K - 1) // (2048 * K)
    g = torch.Generator(device=DEV).manual_seed(K)
    others = plain_others = values = 0
    for _ in range(turns):
        x = torch.randn(M, K, device=DEV, generator=g)
        x = (x * torch.exp(torch.randn(M, 1, device=DEV, generator=g))).bfloat16()
        res = torch.randn(M, K, device=DEV, generator=g).bfloat16()
        weight = (1 + 0.2 * torch.randn(K, device=DEV, generator=g)).bfloat16()
        codes, tiles, _, h = w4.act_rmsnorm(x, weight, form, eps=EPS, residual=res)
        assert torch.equal(h, (x.float() + res.float()).bfloat16())
        eps = float(torch.tensor(EPS, dtype=torch.float32))
        z = h.double() * weight.double()
        y = z / torch.sqrt(h.double().square().mean(1, keepdim=True) + eps)
        e, s = _held(codes, tiles, form)
        we, ws = _exact(y, form)
        other = (e != we) | (s != ws).repeat_interleave(32, 1)
        if other.any():  # each of them lies at a border
            fits = torch.zeros_like(other)
            for d in (-2.0 ** -23, 2.0 ** -23):
                ne, ns = _exact(y * (1 + d), form)
                fits |= (e == ne) & (s == ns).repeat_interleave(32, 1)
            assert fits[other].all()
        others += int(other.sum())
        f = h.float()
        plain = f * weight.float() * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)
        pe, ps = _exact(plain.double(), form)
        plain_others += int(((pe != we) | (ps != ws).repeat_interleave(32, 1)).sum())
        values += y.numel()
    print(f"{form} {K}: {others} of {values} codes differ, {plain_others} of plain fp32's")
    assert others <= 4
    assert plain_others > 4
    assert w4.w4a16_device_status() == 0
