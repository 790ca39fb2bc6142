"""Activations in 4 and 8 bits: what is measured of the operators around the FP4 weights.

Four operators that take the NVFP4 and MXFP4 weights to the block-scaled tensor pipe:

  * ``act_quantize``       BF16 activations into NVFP4, MXFP4 or MXFP8;
  * ``act_rmsnorm``        the residual's addition and the root-mean-square norm in front of it;
  * ``nvfp4_matmul_act``   NVFP4 activations by NVFP4 weights;
  * ``mxfp4_matmul_act``   MXFP4 or MXFP8 activations by MXFP4 weights.

``run`` computes them in plain torch operations in 32 bits, or (``own``) through the framework's
public functions. ``exact`` computes the same in 64 bits from the definition.

Formats. A value is element * block scale (* row or tensor scale):
  * NVFP4: E2M1 elements, an E4M3 scale per 16 and a fp32 scale per row of activations (per tensor
    of weights). With a the row's largest magnitude, at least 2^-80, S = a / 2688; a block's scale
    s is the smallest E4M3 value not below 448 max|block| / a; an element is 2688 x / (s a) rounded
    to the nearest, ties to the even code, at most 6. A block of zeros has scale 0.
  * MXFP4, MXFP8: E2M1 or E4M3 elements, an E8M0 scale 2^X per 32, X = floor(log2 max|block|) - 2
    or - 8 within [-127, 127]; an element is x * 2^-X rounded to the nearest, ties to the even
    code, at most 6 or 448. A block of zeros has the scale's code 0.
Behind a norm x is h * weight / rms, with h the residual rounded to BF16. In NVFP4 1 / rms is the
whole row's and only multiplies S: the codes are those of h * weight.
E2M1 codes lie two in a byte, the even one in the low half. Scales of R rows by C blocks lie in
tiles [ceil(R / 128), ceil(C / 4), 512]: (r, c) at byte (r % 32) 16 + (r / 32 % 4) 4 + c % 4 of tile
(r / 128, c / 4).
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
UP = dict(N=14336, K=4096)         # Llama-3-8B up-projection
DOWN = dict(N=4096, K=14336)       # and its down-projection
QWEN_UP = dict(N=8960, K=1536)     # Qwen2.5-1.5B up-projection


def listed():
    return [
        # the norm in front of a decode step's products: one token, latency is all there is
        {"name": "norm_mxfp8_m1_llama", "op": "norm", "form": "mxfp8", "M": 1, "K": 4096,
         "residual": True},
        # the same norm over a prompt
        {"name": "norm_mxfp8_m4096_llama", "op": "norm", "form": "mxfp8", "M": 4096, "K": 4096,
         "residual": True},
        # the first norm of a small model's ragged batch (no residual yet), rows of a wider array
        {"name": "norm_mxfp8_m203_qwen", "op": "norm", "form": "mxfp8", "M": 203, "K": 1536,
         "residual": False, "wide": 512},
        # the input of the down-projection, a decode batch
        {"name": "quantize_mxfp8_m16_down", "op": "quantize", "form": "mxfp8", "M": 16, "K": 14336},
        # the same of a prompt
        {"name": "quantize_mxfp8_m4096_down", "op": "quantize", "form": "mxfp8", "M": 4096,
         "K": 14336},
        # one token through the up-projection
        {"name": "matmul_nvfp4_m1_up", "op": "matmul", "form": "nvfp4", "M": 1, **UP},
        # a decode batch through the down-projection, 8-bit activations
        {"name": "matmul_mxfp8_m16_down", "op": "matmul", "form": "mxfp8", "M": 16, **DOWN},
        # a ragged batch of a small model
        {"name": "matmul_mxfp4_m300_qwen_up", "op": "matmul", "form": "mxfp4", "M": 300, **QWEN_UP},
        # a prompt through the up-projection
        {"name": "matmul_nvfp4_m4096_up", "op": "matmul", "form": "nvfp4", "M": 4096, **UP},
        # a prompt through the down-projection, 8-bit activations
        {"name": "matmul_mxfp8_m2048_down", "op": "matmul", "form": "mxfp8", "M": 2048, **DOWN},
        # residual, norm and up-projection of a serving batch, as a decoder layer runs them
        {"name": "norm_matmul_nvfp4_m64_up", "op": "norm_matmul", "form": "nvfp4", "M": 64,
         "residual": True, **UP},
        # quantisation and down-projection of a ragged chunk of a prompt
        {"name": "quantize_matmul_mxfp4_m1000_down", "op": "quantize_matmul", "form": "mxfp4",
         "M": 1000, **DOWN},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "matmul", "matmul", "norm_matmul", "quantize_matmul"])
    M = _log(rng, 1, 4096)
    if op in ("norm", "quantize"):
        case = {"op": op, "form": "mxfp8", "M": M, "K": 32 * _log(rng, 8, 448)}
    else:
        form = rng.choice(["nvfp4", "mxfp4", "mxfp8"])
        # an MX product with 8-bit activations takes its weights in boxes of 128
        K = 128 * _log(rng, 2, 112) if form == "mxfp8" else 32 * _log(rng, 8, 448)
        N = 8 * _log(rng, 32, min(1792, 14336 * 4096 // (8 * K)))
        case = {"op": op, "form": form, "M": M, "N": N, "K": K}
    if op != "matmul":
        case["wide"] = rng.choice([0, 0, 512])
    if op.startswith("norm"):
        case["residual"] = rng.random() < 0.7
    return case


def work(case):
    M, K, form = case["M"], case["K"], case["form"]
    bits = {"nvfp4": 4.5, "mxfp4": 4.25, "mxfp8": 8.25}[form]
    wbits = 4.5 if form == "nvfp4" else 4.25
    row = 4 * M if form == "nvfp4" else 0
    bytes_, flops = 0.0, 0.0
    if "norm" in case["op"] or "quantize" in case["op"]:
        bytes_ += 2 * M * K
        flops += 3 * M * K
        if "norm" in case["op"]:
            bytes_ += 2 * K + (4 * M * K if case["residual"] else 0)
            flops += 5 * M * K
    if case["op"] in ("norm", "quantize", "matmul"):
        bytes_ += M * K * bits / 8 + row
    if "matmul" in case["op"]:
        N = case["N"]
        bytes_ += N * K * wbits / 8 + 2 * M * N
        flops += 2 * M * N * K
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------------------------------
# plain forms, in 32 bits
# --------------------------------------------------------------------------------------
def _tiles(s):
    """Scales [rows, cols] (bytes) in tiles; places of no scale hold 0."""
    R, C = s.shape
    rb, cb = (R + 127) // 128, (C + 3) // 4
    t = torch.zeros((rb * 128, cb * 4), dtype=torch.uint8, device=s.device)
    t[:R, :C] = s
    return t.view(rb, 4, 32, cb, 4).permute(0, 3, 2, 1, 4).reshape(rb, cb, 512).contiguous()


def _untile(t, R, C):
    rb, cb, _ = t.shape
    return t.view(rb, cb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cb * 4)[:R, :C]


def _e2m1(v):
    """Codes of the nearest E2M1 values, ties to the even code."""
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    return c + 8 * (v < 0).to(torch.uint8)


def _pack(c):
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _e2m1_value(codes, dtype):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=2).reshape(codes.shape[0], -1).int()
    return grid[c & 7] * (1 - 2 * (c >> 3))


def _e4m3_value(b, dtype):
    return b.view(torch.float8_e4m3fn).to(dtype)


def _e8m0_value(b, dtype):
    return torch.ldexp(torch.ones(b.shape, dtype=dtype, device=b.device), b.int() - 127)


def _quantize(y, form):
    """fp32 [M, K] -> (codes, scales [M, blocks], row scales or None), bytes as they are held."""
    M, K = y.shape
    if form == "nvfp4":
        b = y.view(M, K // 16, 16)
        a = y.abs().amax(1).clamp_min(2.0 ** -80)
        # numerators and denominators under powers of two: exact for BF16 rows, and in range
        ratio = b.abs().amax(2) * (448.0 / 1024.0) / (a / 1024.0)[:, None]
        near = ratio.clamp_max(448.0).to(torch.float8_e4m3fn)
        s = near.view(torch.uint8)
        s = s + ((near.float() < ratio) & (s < 0x7E)).to(torch.uint8)
        den = _e4m3_value(s, torch.float32) * (a / 4096.0)[:, None]
        v = b * (2688.0 / 4096.0) / torch.where(s > 0, den, torch.ones_like(den))[..., None]
        return _pack(_e2m1(v).view(M, K)), s, a / 2688.0
    b = y.view(M, K // 32, 32)
    a = b.abs().amax(2)
    X = (torch.frexp(a)[1] - (3 if form == "mxfp4" else 9)).clamp(-127, 127)
    X = torch.where(a > 0, X, torch.full_like(X, -127))
    v = torch.ldexp(b, -X[..., None]).view(M, K)
    s = (X + 127).to(torch.uint8)
    if form == "mxfp4":
        return _pack(_e2m1(v)), s, None
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), s, None


def _value(codes, scales, form, dtype):
    """What codes and scales [rows, blocks] stand for (without a row's or tensor's scale)."""
    e = _e4m3_value(codes, dtype) if form == "mxfp8" else _e2m1_value(codes, dtype)
    s = _e4m3_value(scales, dtype) if form == "nvfp4" else _e8m0_value(scales, dtype)
    n = 16 if form == "nvfp4" else 32
    return (e.view(e.shape[0], -1, n) * s[..., None]).view(e.shape)


def _rmsnorm(x, residual, weight):
    """(h * weight, 1 / rms per row, h): fp32, fp32 and the new residual in BF16"""
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    f = h.float()
    return f * weight.float(), 1.0 / torch.sqrt(f.square().mean(1) + EPS), h


def _matmul(st, codes, scales, rows):
    """Plain product of activations (codes, scales [M, blocks]) by the state's weights."""
    form, wform = st["form"], "nvfp4" if st["form"] == "nvfp4" else "mxfp4"
    blocks = st["K"] // (16 if form == "nvfp4" else 32)
    a = _value(codes, scales, form, torch.float32)
    w = _value(st["w_codes"], _untile(st["w_scales"], st["N"], blocks), wform, torch.float32)
    y = a @ w.T
    if form == "nvfp4":
        y = y * (rows[:, None] * st["w_scale"])
    return y.bfloat16()


def _plain(st):
    op, form = st["op"], st["form"]
    if op == "matmul":
        blocks = st["K"] // (16 if form == "nvfp4" else 32)
        return (_matmul(st, st["x_codes"], _untile(st["x_scales"], st["M"], blocks),
                        st["x_rows"]),)
    more = ()
    if "norm" in op:
        y, r, h = _rmsnorm(st["x"], st["residual"], st["weight"])
        more = () if st["residual"] is None else (h,)
        codes, scales, rows = _quantize(y if form == "nvfp4" else y * r[:, None], form)
        rows = rows if rows is None else rows * r
    else:
        codes, scales, rows = _quantize(st["x"].float(), form)
    if "matmul" in op:
        return (_matmul(st, codes, scales, rows),) + more
    return (codes.view(torch.float8_e4m3fn), _tiles(scales).view(torch.float8_e8m0fnu)) + more


# --------------------------------------------------------------------------------------
# the framework's functions
# --------------------------------------------------------------------------------------
def _framework(st):
    import gemv_w4a16_group_gb300 as g

    op, form = st["op"], st["form"]
    more = ()
    if op == "matmul":
        codes, scales, rows = st["x_codes"], st["x_scales"], st["x_rows"]
    else:
        keep = dict(codes=st["codes"], scales=st["scales"], row_scales=st["rows"])
        if "norm" in op:
            codes, scales, rows, h = g.act_rmsnorm(
                st["x"], st["weight"], form, eps=EPS, residual=st["residual"],
                residual_out=st["residual_out"], **keep)
            more = () if h is None else (h,)
        else:
            codes, scales, rows = g.act_quantize(st["x"], form, **keep)
        if "matmul" not in op:
            return (codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)) + more
    if form == "nvfp4":
        y = g.nvfp4_matmul_act(codes, scales, rows, st["w_codes"], st["w_scales"], st["w_scale"])
    else:
        y = g.mxfp4_matmul_act(codes, scales, st["w_codes"], st["w_scales"])
    return (y,) + more


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _activations(g, M, K):
    """BF16 rows with a few channels far above the others and tokens of different size."""
    chan = torch.where(torch.rand(K, device=DEV, generator=g) < 0.01, 12.0, 1.0)
    size = torch.exp(0.5 * torch.randn(M, 1, device=DEV, generator=g))
    return (torch.randn(M, K, device=DEV, generator=g) * chan * size).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, form, M, K = case["op"], case["form"], case["M"], case["K"]
    st = dict(case)
    x = _activations(g, M, K)
    if case.get("wide"):  # rows that lie in a wider array, as a fused projection leaves them
        full = torch.zeros(M, K + case["wide"], dtype=torch.bfloat16, device=DEV)
        full[:, :K] = x
        x = full[:, :K]
    if "matmul" in op:
        N, wform = case["N"], "nvfp4" if form == "nvfp4" else "mxfp4"
        w = torch.randn(N, K, device=DEV, generator=g)
        w *= 0.02 * torch.exp(0.3 * torch.randn(N, 1, device=DEV, generator=g))
        if wform == "nvfp4":  # one scale for the tensor
            codes, s, S = _quantize(w.view(1, N * K), wform)
            st["w_codes"], s, st["w_scale"] = codes.view(N, K // 2), s.view(N, -1), S
        else:
            st["w_codes"], s, _ = _quantize(w, wform)
        st["w_scales"] = _tiles(s)
        del w
    if op == "matmul":
        st["x_codes"], s, st["x_rows"] = _quantize(x.float(), form)
        st["x_scales"] = _tiles(s)
        return st
    st["x"] = x
    if "norm" in op:
        st["weight"] = (1 + 0.2 * torch.randn(K, device=DEV, generator=g)).bfloat16()
        st["residual"] = (4 * _activations(g, M, K).float()).bfloat16() if case["residual"] else None
        st["residual_out"] = torch.empty_like(x) if case["residual"] else None
    # a decode loop keeps the buffers between the norm and the product
    n = 16 if form == "nvfp4" else 32
    st["codes"] = torch.empty(M, K if form == "mxfp8" else K // 2, dtype=torch.uint8, device=DEV)
    st["scales"] = _tiles(torch.zeros(M, K // n, dtype=torch.uint8, device=DEV))
    st["rows"] = torch.empty(M, device=DEV) if form == "nvfp4" else None
    return st


# --------------------------------------------------------------------------------------
# 64 bits, from the definition
# --------------------------------------------------------------------------------------
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1_near64(v):
    """Nearest E2M1 value of each of v (64 bits): among the grid's values the one at the smallest
    distance, of two the one with the even code."""
    a = v.abs().clamp_max(6.0)
    best = torch.zeros_like(a)
    gap = a.clone()
    for i, x in enumerate(_GRID[1:], 1):
        d = (a - x).abs()
        take = (d < gap) | ((d == gap) & (i % 2 == 0))
        best = torch.where(take, torch.full_like(a, x), best)
        gap = torch.where(take, d, gap)
    return torch.copysign(best, v)


def _e4m3_near64(v, up=False):
    """E4M3 values of v (64 bits): nearest, ties to even, or the next one not below; at most 448."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    # log2 of a power of two may come out short by a rounding
    step = torch.where(a >= 16 * step, 2 * step, step)
    q = torch.ceil(a / step) if up else torch.round(a / step)
    return torch.copysign((q * step).clamp_max(448.0), v)


def _scale_exponent64(a, top):
    m, e = torch.frexp(a)
    X = (e - 1 - top).clamp(-127, 127).to(a.dtype)
    return torch.where(a > 0, X, torch.full_like(X, -127.0))


def _quantize64(y, form):
    """(elements, scales [M, blocks], row scales) as values"""
    M, K = y.shape
    if form == "nvfp4":
        b = y.reshape(M, K // 16, 16)
        a = y.abs().amax(1).clamp_min(2.0 ** -80)
        s = _e4m3_near64(448.0 * b.abs().amax(2) / a[:, None], up=True)
        den = torch.where(s > 0, s * a[:, None], torch.ones_like(s))
        e = _e2m1_near64(2688.0 * b / den[..., None])
        return torch.where(s[..., None] > 0, e, 0.0).reshape(M, K), s, a / 2688.0
    b = y.reshape(M, K // 32, 32)
    X = _scale_exponent64(b.abs().amax(2), 2 if form == "mxfp4" else 8)
    s = torch.exp2(X)
    v = b / s[..., None]
    e = _e2m1_near64(v) if form == "mxfp4" else _e4m3_near64(v)
    return e.reshape(M, K), s, None


def _spread64(e, s):
    return (e.reshape(s.shape[0], s.shape[1], -1) * s[..., None]).reshape(e.shape)


def _e8m0_64(b):
    return torch.exp2(b.double() - 127.0)


def _elements64(codes):
    table = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float64, device=DEV)
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=DEV)
    out[:, 0::2] = table[(codes & 15).long()]
    out[:, 1::2] = table[(codes >> 4).long()]
    return out


def _held64(codes, tiles, rows, cols, form):
    """Values of what is held in codes and scale tiles (without a row's or tensor's scale)."""
    r = torch.arange(rows, device=DEV)[:, None]
    c = torch.arange(cols, device=DEV)[None, :]
    at = ((r // 128 * tiles.shape[1] + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4)
    b = tiles.reshape(-1)[at]
    s = b.view(torch.float8_e4m3fn).double() if form == "nvfp4" else _e8m0_64(b)
    e = codes.view(torch.float8_e4m3fn).double() if form == "mxfp8" else _elements64(codes)
    return _spread64(e, s)


def exact(case, seed):
    st = prepare(case, seed)
    op, form, M, K = case["op"], case["form"], case["M"], case["K"]
    cols = K // (16 if form == "nvfp4" else 32)
    more = ()
    if op == "matmul":
        a = _held64(st["x_codes"], st["x_scales"], M, cols, form)
        if form == "nvfp4":
            a *= st["x_rows"].double()[:, None]
    else:
        y = st["x"].double()
        if "norm" in op:
            if case["residual"]:
                # the sum is rounded to BF16, and the norm is that of the rounded residual
                h = (y + st["residual"].double()).float().bfloat16().double()
                more, y = (h,), h
            rms = torch.sqrt((y * y).sum(1, keepdim=True) / K + EPS)
            y = y * st["weight"].double()
            if form == "nvfp4":
                e, s, S = _quantize64(y, form)
                S = S / rms[:, 0]
            else:
                e, s, S = _quantize64(y / rms, form)
        else:
            e, s, S = _quantize64(y, form)
        if "matmul" not in op:
            t = torch.zeros((M + 127) // 128, (cols + 3) // 4, 512, dtype=torch.float64, device=DEV)
            t += 2.0 ** -127  # places of no scale hold the code 0
            r = torch.arange(M, device=DEV)[:, None]
            c = torch.arange(cols, device=DEV)[None, :]
            t[r // 128, c // 4, r % 32 * 16 + r // 32 % 4 * 4 + c % 4] = s
            return (e, t) + more
        a = _spread64(e, s)
        if form == "nvfp4":
            a *= S[:, None]
    w = _held64(st["w_codes"], st["w_scales"], case["N"], cols, "nvfp4" if form == "nvfp4" else "mxfp4")
    y = a @ w.T
    if form == "nvfp4":
        y *= st["w_scale"].double()
    return (y,) + more
