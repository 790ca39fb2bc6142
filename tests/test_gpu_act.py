"""Activations in 4 and 8 bits on the GPU against tests/act_reference.py (64 bits).

Bounds, before any run:
  * codes and scales of BF16 rows are exact: MX scales are powers of two; NVFP4's quotients have
    numerators of at most 13 and denominators of at most 12 significant bits, so one that is not a
    border of E2M1 or E4M3 (at most 5 bits) is at least 2^-18 of itself from it, and fp32's quotient
    is within 2^-23;
  * the norm's h is exact, and so are NVFP4's codes and block scales (h * weight has 16 bits).
    1 / rms is off by at most D = 2^-20 of itself: a thread adds at most 64 squares and the
    threads join in 10 steps, all terms positive, 74 roundings of 2^-24 at worst, halved by the
    root, and three more; MX codes and scales are those of some y (1 + d), |d| <= D;
  * a product: codes times scales are exact; each MMA (32 or 64 values of k) adds with at most
    2^-22 of the sum A of its terms' magnitudes, so K / 32 of them with K 2^-27 A; a row's and a
    tensor's scale 2 * 2^-24 of the value; the rounding to BF16 2^-8 of it."""
import numpy as np
import pytest
import torch

import act_reference as ref

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"
FORMS = ["nvfp4", "mxfp4", "mxfp8"]
EPS = 1e-6
D = 2.0 ** -20


def _ok():
    assert w4.w4a16_device_status() == 0


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rows(M, K, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))
    return (x * torch.where(torch.rand(K, generator=g) < 0.02, 15.0, 1.0)).bfloat16()


def _held(codes, scales, form, K):
    """(elements, scales [M, blocks]) as values"""
    b = ref.untile(scales.cpu().numpy(), codes.shape[0], K // ref.BLOCK[form])
    return ref.element_values(codes.cpu().numpy(), form), ref.scale_values(b, form)


def _check_exact(got, want, row_tol=2.0 ** -23):
    (e, s), r, (we, ws, wr) = got[0], got[1], want
    assert np.array_equal(s, ws), "block scales"
    assert np.array_equal(e, we), "codes"
    if wr is not None:
        assert (np.abs(_f64(r) - wr) <= row_tol * wr).all(), "row scales"


def _quantized(x, form, **kw):
    c, s, r = w4.act_quantize(x, form, **kw)
    return (_held(c, s, form, x.shape[1]), r), (c, s, r)


def _special(M, K, seed):
    """Zeros, ties, subnormals and both ends of BF16's range."""
    x = _rows(M, K, seed).float().numpy()
    x[0] = 0
    if M > 1:
        x[1, :16] = -0.0
        x[1, 16:32] = 0
    if M > 2:  # quotients on the grid's borders: blocks whose largest value is 6
        x[2] = np.resize([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5,
                          -3.5, -5, 0.125], K)
    if M > 3:
        x[3] *= 2.0 ** -120   # block scales that meet E8M0's lower end, rows below 2^-80
        x[3, : K // 2] = np.resize([2.0 ** -133, 0, -(2.0 ** -130), 2.0 ** -126], K // 2)
    if M > 4:
        x[4] = np.resize([3.38e38, 1e30, -1e38, 1e20, 1, 3e38, -2e37, 5e36], K)
    if M > 5:
        x[5, 0] = 1e30        # the rest of the row far below one value
    if M > 6:  # MXFP8's borders: halves between E4M3 values, and past 448
        x[6] = np.resize([448, 464, 472, 480, 1.0625, 1.1875, 17, 19, 0.0009765625, 0.0029296875,
                          -464, -17, 500, 2 ** -10, 3 * 2.0 ** -11, 31], K)
    return torch.from_numpy(x).bfloat16()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M,K", [(1, 32), (7, 64), (33, 96), (2, 1536), (130, 416), (5, 14336),
                                 (9, 8960), (3, 16384), (2, 65536), (257, 2080)])
def test_quantize_is_exact(form, M, K):
    x = _special(M, K, 3 * M + K)
    got, _ = _quantized(x.to(DEV), form)
    want = ref.quantize(_f64(x), form)
    if form == "nvfp4" and M > 3:
        # a row below 2^-80: its quotients' numerators may be subnormal in fp32, off by 2^-149 of
        # a value that is 2^-90 at least in units of the smallest code, so still exact
        assert want[2][3] >= 2.0 ** -92
    _check_exact(got, want)
    _ok()


@pytest.mark.parametrize("form", FORMS)
def test_quantize_takes_rows_of_a_wider_array(form):
    M, K = 37, 352
    wide = _rows(M, 3 * K + 8, 1).to(DEV)
    x = wide[:, K:2 * K]
    got, _ = _quantized(x, form)
    _check_exact(got, ref.quantize(_f64(x), form))
    one, _ = _quantized(wide[5:6, K:2 * K], form)
    _check_exact(one, ref.quantize(_f64(wide[5:6, K:2 * K]), form))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M,K", [(5, 32), (127, 160), (129, 1056)])
def test_quantize_leaves_other_rows_alone(form, M, K):
    """Scale words of rows past M keep what they held; those of the rows are whole (0 past the
    last block)."""
    x = _rows(M, K, 5).to(DEV)
    blocks = K // ref.BLOCK[form]
    tiles = torch.full(((M + 127) // 128, (blocks + 3) // 4, 512), 0xA5, dtype=torch.uint8,
                       device=DEV)
    w4.act_quantize(x, form, scales=tiles)
    padded = ref.untile(tiles.cpu().numpy(), tiles.shape[0] * 128, tiles.shape[1] * 4)
    assert (padded[M:] == 0xA5).all()
    assert (padded[:M, blocks:] == 0).all()
    assert (ref.scale_values(padded[:M, :blocks], form) == ref.quantize(_f64(x), form)[1]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_make_their_row_nan(form, bad):
    M, K, N = 9, 256, 40
    x = _rows(M, K, 6).to(DEV)
    x[4, 70] = bad
    _, (c, s, r) = _quantized(x, form)
    y = _matmul(form, (c, s, r), _weights(form, N, K, 7))
    want = torch.zeros(M, dtype=torch.bool, device=DEV)
    want[4] = True
    assert torch.equal(y.isnan().all(1), want) and torch.equal(y.isnan().any(1), want)
    clean = x.clone()
    clean[4] = 0
    keep = _matmul(form, w4.act_quantize(clean, form), _weights(form, N, K, 7))
    assert torch.equal(y[~want], keep[~want]), "other rows do not change"
    c, s, r, _ = w4.act_rmsnorm(x, torch.ones(K, device=DEV).bfloat16(), form)
    y = _matmul(form, (c, s, r), _weights(form, N, K, 7))
    assert torch.equal(y.isnan().all(1), want) and torch.equal(y.isnan().any(1), want)
    _ok()


def _check_norm(form, out, x, residual, weight, K, eps=EPS):
    c, s, r, h = out
    z, rinv, want_h = ref.rmsnorm(_f64(x), None if residual is None else _f64(residual),
                                  _f64(weight), eps)
    if residual is None:
        assert h is None
    else:
        assert np.array_equal(_f64(h), want_h)
    e, sv = _held(c, s, form, K)
    if form == "nvfp4":
        we, ws, wr = ref.quantize(z, form)
        _check_exact(((e, sv), r), (we, ws, wr * rinv), 2 * D)
        return
    fits = None
    for d in (-D, 0, D):
        we, ws, _ = ref.quantize(z * rinv[:, None] * (1 + d), form)
        n = ref.BLOCK[form]
        same = (e == we) & (np.repeat(sv, n, 1) == np.repeat(ws, n, 1))
        fits = same if fits is None else fits | same
    assert fits.all(), f"{(~fits).sum()} of {fits.size} values"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (1, 4096), (34, 1536), (130, 448), (6, 14336),
                                 (2, 65536)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_rmsnorm(form, M, K, with_residual):
    g = torch.Generator().manual_seed(M + K)
    x = _rows(M, K, M + K).to(DEV)
    res = (3 * _rows(M, K, M + K + 1)).to(DEV) if with_residual else None
    weight = (1 + 0.3 * torch.randn(K, generator=g)).bfloat16().to(DEV)
    before = None if res is None else res.clone()
    out = w4.act_rmsnorm(x, weight, form, eps=EPS, residual=res)
    _check_norm(form, out, x, res, weight, K)
    assert res is None or torch.equal(res, before), "the residual itself stays"
    _ok()


@pytest.mark.parametrize("form", FORMS)
def test_rmsnorm_in_place_and_strided(form):
    M, K = 19, 608
    weight = torch.linspace(-1, 2, K).bfloat16().to(DEV)
    wide = _rows(M, 2 * K, 8).to(DEV)
    x, res = wide[:, K:], (2 * _rows(M, K + 16, 9)).bfloat16().to(DEV)
    r0, x0 = res[:, :K].clone(), x.clone()
    out = w4.act_rmsnorm(x, weight, form, residual=res[:, :K], residual_out=res[:, :K])
    assert out[3].data_ptr() == res.data_ptr()
    _check_norm(form, out, x0, r0, weight, K)
    out = w4.act_rmsnorm(x, weight, form, residual=r0, residual_out=x)
    _check_norm(form, out, x0, r0, weight, K)
    assert torch.equal(wide[:, K:], out[3])


@pytest.mark.parametrize("form", FORMS)
def test_rmsnorm_rows_of_zeros_and_small_and_large_ones(form):
    K = 256
    x = _rows(5, K, 10).float()
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 50
    x[3] = 0
    x[3, 17] = 1e-3
    x, weight = x.bfloat16().to(DEV), _rows(1, K, 11)[0].to(DEV)
    for eps in (1e-5, 1e-30):
        _check_norm(form, w4.act_rmsnorm(x, weight, form, eps=eps), x, None, weight, K,
                    float(np.float32(eps)))
    # squares past fp32's range
    big = torch.full((1, K), 1e30, device=DEV).bfloat16()
    y = _matmul(form, w4.act_rmsnorm(big, weight, form)[:3], _weights(form, 8, K, 1))
    assert y.isnan().all()


# ---- products ------------------------------------------------------------------------------
def _weights(form, N, K, seed):
    """(codes, scale tiles, tensor scale or None, what they stand for in 64 bits on the GPU)"""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randn(N, K, device=DEV, generator=g) * 0.03
    w *= torch.exp(0.5 * torch.randn(N, 1, device=DEV, generator=g))
    if form == "nvfp4":
        pad = (-K) % 128  # nvfp4_quantize takes whole 128s: the rows' ends are cut off again
        wide = torch.nn.functional.pad(w, (0, pad))
        codes, scales, S = w4.nvfp4_quantize(wide)
        codes, scales = codes[:, :K // 2].contiguous(), scales[:, :K // 16].contiguous()
        held = ref.values(codes.cpu().numpy(), scales.cpu().numpy(), form) * _f64(S)
    else:
        codes, scales = w4.mxfp4_quantize(w)
        S = None
        held = ref.values(codes.cpu().numpy(), scales.cpu().numpy(), "mxfp4")
    return codes, w4.fp4_prepare_scales(scales), S, torch.from_numpy(held).to(DEV)


def _matmul(form, x, weights, **kw):
    if form == "nvfp4":
        return w4.nvfp4_matmul_act(x[0], x[1], x[2], weights[0], weights[1], weights[2], **kw)
    return w4.mxfp4_matmul_act(x[0], x[1], weights[0], weights[1], **kw)


def _x_held(form, x, K):
    e, s = _held(x[0], x[1], form, K)
    v = (e.reshape(e.shape[0], s.shape[1], -1) * s[..., None]).reshape(e.shape)
    if form == "nvfp4":
        v = v * _f64(x[2])[:, None]
    return torch.from_numpy(v).to(DEV)


def _check_product(y, xh, wh, K):
    want = xh @ wh.T
    terms = xh.abs() @ wh.abs().T
    tol = 2.0 ** -8 * want.abs() + (K * 2.0 ** -27 + 2.0 ** -22) * terms
    off = (y.double() - want).abs()
    assert (off <= tol).all(), f"{int((off > tol).sum())} of {off.numel()}, worst {(off / tol).max()}"


SHAPES = [(1, 8, 128), (1, 1, 256), (3, 40, 32), (2, 129, 96), (16, 333, 288), (17, 128, 384),
          (32, 257, 640), (33, 1000, 1536), (64, 130, 1664), (65, 384, 256), (127, 200, 512),
          (128, 127, 4096), (129, 264, 544), (200, 1001, 768), (256, 256, 1024), (257, 520, 8960),
          (300, 96, 14336), (511, 640, 256), (1000, 1536, 1536), (1, 4096, 14336),
          (1, 14336, 4096), (640, 8960, 128)]


@pytest.mark.parametrize("form,M,N,K", [(f, *s) for f in FORMS for s in SHAPES
                                        if f != "mxfp8" or s[2] % 128 == 0])
def test_product(form, M, N, K):
    x = w4.act_quantize(_rows(M, K, M + N).to(DEV), form)
    w = _weights(form, N, K, N + K)
    y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    _matmul(form, x, w, y=y[:M])
    _ok()
    _check_product(y[:M], _x_held(form, x, K), w[3], K)
    assert (y[M] == 7).all(), "the row behind the last is left as it was"


@pytest.fixture(params=[1, 2, 3, 4], ids=["narrow", "pairs", "pairs-2", "pairs-4"])
def forced(request):
    """Each kernel of the products at sizes that the choice by size may give to another."""
    prev = w4.testing_set_act_kernel(request.param)
    yield request.param
    w4.testing_set_act_kernel(prev)


@pytest.mark.parametrize("form,M,N,K", [(f, *s) for f in FORMS for s in
                                        [(1, 8, 128), (5, 129, 384), (100, 1001, 640),
                                         (129, 264, 256), (256, 520, 1152), (257, 256, 2048),
                                         (520, 1288, 512), (1100, 4096, 128), (700, 136, 4096),
                                         (2100, 6144, 1024)]])
def test_product_of_each_kernel(forced, form, M, N, K):
    x = w4.act_quantize(_rows(M, K, M + N).to(DEV), form)
    w = _weights(form, N, K, N + K)
    y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    _matmul(form, x, w, y=y[:M])
    _ok()
    _check_product(y[:M], _x_held(form, x, K), w[3], K)
    assert (y[M] == 7).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M", [1, 5, 130, 700])
def test_product_ignores_what_lies_past_its_rows(form, M):
    """Scale words past M and past the last weight row hold NaN."""
    N, K = 200, 384
    x = list(w4.act_quantize(_rows(M, K, 1).to(DEV), form))
    w = list(_weights(form, N, K, 2))
    y0 = _matmul(form, x, w)
    for i, (t, rows) in ((0, (x, M)), (1, (w, N))):
        tiles = t[1].cpu().numpy().copy()
        R = np.arange(rows, tiles.shape[0] * 128)[:, None]
        C = np.arange(tiles.shape[1] * 4)[None]
        tiles[R // 128, C // 4, R % 32 * 16 + R // 32 % 4 * 4 + C % 4] = 0xFF
        t[1] = torch.from_numpy(tiles).to(DEV)
    assert torch.equal(_matmul(form, x, w), y0)


@pytest.mark.parametrize("form", FORMS)
def test_product_does_not_depend_on_other_rows_of_a_call(form):
    """Rows of a batch equal the same rows under other neighbours."""
    M, N, K = 90, 300, 1024
    x = _rows(M, K, 3).to(DEV)
    w = _weights(form, N, K, 4)
    y = _matmul(form, w4.act_quantize(x, form), w)
    x2 = x.flip(0).contiguous()
    y2 = _matmul(form, w4.act_quantize(x2, form), w)
    assert torch.equal(y, y2.flip(0))


@pytest.mark.parametrize("form", FORMS)
def test_product_is_the_same_every_time(form):
    for M, N, K in [(4, 4096, 2048), (700, 1000, 1024)]:
        x = w4.act_quantize(_rows(M, K, 3).to(DEV), form)
        w = _weights(form, N, K, 4)
        y = _matmul(form, x, w)
        for _ in range(5):
            assert torch.equal(y, _matmul(form, x, w))


@pytest.mark.parametrize("form", FORMS)
def test_extreme_scales(form):
    """Blocks 2^60 apart, and scales at both ends of their range, next to blocks of zeros."""
    M, N, K = 24, 136, 512
    x = _rows(M, K, 12).float()
    e = torch.arange(K // 32) % 7 - 3
    x *= torch.repeat_interleave(2.0 ** (10.0 * e), 32)
    x[3] = 0
    x[5, 64:] = 0
    x = w4.act_quantize(x.bfloat16().to(DEV), form)
    w = _weights(form, N, K, 13)
    _check_product(_matmul(form, x, w), _x_held(form, x, K), w[3], K)


@pytest.mark.parametrize("form", FORMS)
def test_offsets_past_32_bits(form):
    """More than 2^31 values of x and of y, 2^32 bytes of each in BF16."""
    M, K, N = 280_000, 8192, 8192
    g = torch.Generator(device=DEV).manual_seed(1)
    few = torch.randn(1000, K, device=DEV, generator=g).bfloat16()
    x = few.repeat(M // 1000, 1)
    q = w4.act_quantize(x, form)
    del x
    first = w4.act_quantize(few[-200:], form)
    assert torch.equal(q[0][-200:], first[0])
    w = _weights(form, N, K, 2)
    y = _matmul(form, q, w)
    _ok()
    _check_product(y[-200:], _x_held(form, first, K), w[3], K)
    assert torch.equal(y[-1000:], y[:1000])


# ---- streams, graphs, and the operators together ---------------------------------------------
@pytest.mark.parametrize("form", FORMS)
def test_streams_and_graphs(form):
    """A step (norm, product) on another stream, as a raw handle, and captured and replayed with
    new inputs in the same buffers; two captured steps replayed at once."""
    K, N = 512, 640
    weight = torch.ones(K, device=DEV).bfloat16()
    w = _weights(form, N, K, 5)

    def step(x, res, stream=None):
        c, s, r, h = w4.act_rmsnorm(x, weight, form, residual=res, stream=stream)
        return _matmul(form, (c, s, r), w, stream=stream), h

    def want(M, seed):
        y, h = step(_rows(M, K, seed).to(DEV), _rows(M, K, seed + 1).to(DEV))
        torch.cuda.synchronize()
        return y, h

    stream = torch.cuda.Stream()
    graphs = []
    for M in (3, 200):
        x, res = _rows(M, K, 20).to(DEV), _rows(M, K, 21).to(DEV)
        torch.cuda.synchronize()
        for handle in (stream, stream.cuda_stream):
            y, h = step(x, res, handle)
            stream.synchronize()
            y0, h0 = want(M, 20)
            assert torch.equal(y, y0) and torch.equal(h, h0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step(x, res)
        graphs.append((graph, x, res, out, M))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (30, 40):
        expect = []
        for graph, x, res, out, M in graphs:
            expect.append(want(M, seed + M))
            x.copy_(_rows(M, K, seed + M))
            res.copy_(_rows(M, K, seed + M + 1))
        torch.cuda.synchronize()
        for _ in range(3):
            for (graph, *_), st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        for (graph, x, res, out, M), (y, h) in zip(graphs, expect):
            assert torch.equal(out[0], y) and torch.equal(out[1], h)
    _ok()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 1024), (64, 14336, 1024), (128, 14336, 1024),
                                   (128, 1024, 7168), (300, 4096, 1024)])
def test_long_chains_in_graphs(form, M, N, K):
    """Norm and product twenty times in one graph, on two sets of buffers in turn, replayed a
    hundred times without a pause: kernels that begin before the last one has ended must leave
    it, and one another, the SMs that they need."""
    weight = torch.ones(K, device=DEV).bfloat16()
    w = _weights(form, N, K, 6)
    states = []
    for seed in (60, 70):
        x, res = _rows(M, K, seed).to(DEV), _rows(M, K, seed + 1).to(DEV)
        states.append((x, res, torch.empty_like(res), w4.act_quantize(x, form)))

    def step(x, res, out, q):
        c, s, r, _ = w4.act_rmsnorm(x, weight, form, residual=res, residual_out=out, codes=q[0],
                                    scales=q[1], row_scales=q[2])
        return _matmul(form, (c, s, r), w)

    want = [step(*st).clone() for st in states]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [step(*states[i % 2]) for i in range(20)]
    for _ in range(100):
        graph.replay()
    torch.cuda.synchronize()
    _ok()
    for i, y in enumerate(outs):
        assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("calls", [
    [("nvfp4", 64, 14336, 1024), ("mxfp8", 8, 4096, 4096), ("mxfp4", 512, 4096, 8192)],
    [("nvfp4", 300, 4096, 4096), ("nvfp4", 17, 14336, 2048), ("mxfp8", 64, 4096, 7168)],
    [("mxfp4", 128, 1536, 8960), ("mxfp8", 1000, 2048, 2048), ("nvfp4", 1, 4096, 4096)],
])
def test_chains_on_three_streams(calls):
    """Graphs of norms and products on three streams at once: pairs, clusters of pairs and
    clusters of single CTAs want the same SMs, and every one of them gets them."""
    runs = []
    for form, M, N, K in calls:
        weight = torch.ones(K, device=DEV).bfloat16()
        w = _weights(form, N, K, 6)
        states = []
        for seed in (60, 70):
            x, res = _rows(M, K, seed).to(DEV), _rows(M, K, seed + 1).to(DEV)
            states.append((x, res, torch.empty_like(res), w4.act_quantize(x, form)))

        def step(x, res, out, q):
            c, s, r, _ = w4.act_rmsnorm(x, weight, form, residual=res, residual_out=out,
                                        codes=q[0], scales=q[1], row_scales=q[2])
            return _matmul(form, (c, s, r), w)

        want = [step(*st).clone() for st in states]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [step(*states[i % 2]) for i in range(20)]
        runs.append((graph, outs, want, torch.cuda.Stream(), (weight, w, states)))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, _, _, stream, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    _ok()
    for _, outs, want, _, _ in runs:
        for i, y in enumerate(outs):
            assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M", [1, 6, 150])
def test_a_layer_as_it_is_used(form, M):
    """Residual and norm, the up and gate projections, their product quantized, the down
    projection, and the next norm with its residual: each step against 64 bits from what the
    step before it left."""
    K, F = 512, 1408
    weight = (1 + 0.1 * torch.randn(K)).bfloat16().to(DEV)
    up, down = _weights(form, 2 * F, K, 1), _weights(form, K, F, 2)
    x, res = _rows(M, K, 50).to(DEV), _rows(M, K, 51).to(DEV)
    out = w4.act_rmsnorm(x, weight, form, residual=res)
    _check_norm(form, out, x, res, weight, K)
    both = _matmul(form, out[:3], up)
    _check_product(both, _x_held(form, out, K), up[3], K)
    act = (torch.nn.functional.silu(both[:, :F].float()) * both[:, F:].float()).bfloat16()
    q = w4.act_quantize(act, form)
    _check_exact((_held(q[0], q[1], form, F), q[2]), ref.quantize(_f64(act), form))
    y = _matmul(form, q, down)
    _check_product(y, _x_held(form, q, F), down[3], F)
    out2 = w4.act_rmsnorm(y, weight, form, residual=out[3], residual_out=out[3])
    z, rinv, h = ref.rmsnorm(_f64(y), ref.rmsnorm(_f64(x), _f64(res), _f64(weight), EPS)[2],
                             _f64(weight), EPS)
    assert np.array_equal(_f64(out2[3]), h)
    _ok()


def test_prepared_scales_are_the_weights_scales():
    for N, C in [(1, 1), (127, 3), (129, 8), (300, 257)]:
        s = torch.randint(0, 256, (N, C), dtype=torch.uint8, device=DEV)
        t = w4.fp4_prepare_scales(s)
        full = ref.untile(t.cpu().numpy(), t.shape[0] * 128, t.shape[1] * 4)
        assert np.array_equal(full[:N, :C], s.cpu().numpy())
        assert (full[N:] == 0).all() and (full[:, C:] == 0).all()


def test_python_refusals():
    x = _rows(4, 64, 1).to(DEV)
    w = torch.ones(64, device=DEV).bfloat16()
    with pytest.raises(ValueError, match="format"):
        w4.act_quantize(x, "fp8")
    with pytest.raises(TypeError, match="x must be"):
        w4.act_quantize(x.float())
    with pytest.raises(ValueError, match="CUDA"):
        w4.act_quantize(x.cpu())
    with pytest.raises(ValueError, match="dense rows"):
        w4.act_quantize(x.t().contiguous().t())
    with pytest.raises(ValueError, match="row scales"):
        w4.act_quantize(x, "mxfp4", row_scales=torch.empty(4, device=DEV))
    with pytest.raises(ValueError, match="codes"):
        w4.act_quantize(x, "mxfp8", codes=torch.empty(4, 32, dtype=torch.uint8, device=DEV))
    with pytest.raises(w4.W4A16Error, match="INVALID"):
        w4.act_quantize(x[:, :40])
    with pytest.raises(w4.W4A16Error, match="MISALIGNED"):
        w4.act_quantize(_rows(1, 72, 1).to(DEV)[:, 4:36])
    with pytest.raises(ValueError, match="residual_out needs"):
        w4.act_rmsnorm(x, w, residual_out=x)
    with pytest.raises(ValueError, match="weight"):
        w4.act_rmsnorm(x, w[:32].contiguous())
    with pytest.raises(ValueError, match="residual must be"):
        w4.act_rmsnorm(x, w, residual=x[:3])
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(w4.W4A16Error, match="INVALID"):
            w4.act_rmsnorm(x, w, eps=eps)
    q = w4.act_quantize(x, "mxfp4")
    wt = _weights("mxfp4", 16, 64, 1)
    with pytest.raises(ValueError, match="x_codes"):
        w4.mxfp4_matmul_act(q[0][:, :16].contiguous(), q[1], wt[0], wt[1])
    with pytest.raises(w4.W4A16Error, match="INVALID"):  # 8-bit activations: whole 128s
        q8 = w4.act_quantize(x, "mxfp8")
        w4.mxfp4_matmul_act(q8[0], q8[1], wt[0], wt[1])
    with pytest.raises(ValueError, match="scale_tiles"):
        w4.mxfp4_matmul_act(q[0], q[1], wt[0], wt[1][:, :0])
    torch.cuda.synchronize()
    _ok()
