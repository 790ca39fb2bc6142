"""Pairs of CTAs among other kernels' CTAs: products and norms on many streams at once, each stream's
results those of the stream alone. (A pair's CTAs may begin at different times where other kernels'
CTAs leave their SMs.)"""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"


def _chain(form, M, N, K, kernel):
    """A step (norm, product by the given kernel) on buffers of its own."""
    g = torch.Generator(device=DEV).manual_seed(M + N + K)

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    x, res, weight = randn(M, K).bfloat16(), randn(M, K).bfloat16(), randn(K).bfloat16()
    out = torch.empty_like(res)
    if form == "nvfp4":
        codes, scales, S = w4.nvfp4_quantize(randn(N, K))
    else:
        codes, scales = w4.mxfp4_quantize(randn(N, K))
    tiles = w4.fp4_prepare_scales(scales)

    def step():
        c, s, r, _ = w4.act_rmsnorm(x, weight, form, residual=res, residual_out=out)
        prev = w4.testing_set_act_kernel(kernel)
        try:
            if form == "nvfp4":
                return w4.nvfp4_matmul_act(c, s, r, codes, tiles, S)
            return w4.mxfp4_matmul_act(c, s, codes, tiles)
        finally:
            w4.testing_set_act_kernel(prev)
    return step


@pytest.mark.parametrize("calls", [
    # pairs alone, two and four a tile, and clusters of single CTAs
    [("nvfp4", 300, 4096, 1024, 2), ("mxfp4", 500, 2048, 4096, 3), ("mxfp8", 200, 1032, 4096, 4),
     ("nvfp4", 9, 4096, 4096, 1)],
    # pairs among pairs, and prompts' norms
    [("nvfp4", 64, 14336, 512, 2), ("mxfp4", 64, 14336, 512, 2), ("mxfp8", 64, 8192, 512, 2),
     ("mxfp8", 1500, 256, 4096, 2)],
    # fours of pairs among clusters of eight
    [("mxfp4", 256, 2048, 4096, 4), ("nvfp4", 256, 2048, 4096, 4), ("nvfp4", 33, 2048, 8192, 1),
     ("mxfp8", 16, 4096, 8192, 1)]])
@pytest.mark.parametrize("graphs", [True, False])
def test_pairs_among_other_kernels(calls, graphs):
    chains = []
    for call in calls:
        step = _chain(*call)
        want = step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        if graphs:
            with torch.cuda.graph(graph):
                outs = [step() for _ in range(20)]
        else:
            outs = [None] * 20
        chains.append((step, want, graph, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(200 if graphs else 5):
        for i in range(1 if graphs else 20):
            for step, _, graph, outs, stream in chains:
                with torch.cuda.stream(stream):
                    if graphs:
                        graph.replay()
                    else:
                        outs[i] = step()
    # a standstill becomes a failure here: no wait of the host without a limit
    ends = []
    for *_, stream in chains:
        ends.append(torch.cuda.Event())
        ends[-1].record(stream)
    until = time.monotonic() + 60
    while not all(e.query() for e in ends):
        assert time.monotonic() < until, "the chains stand still"
        time.sleep(0.001)
    assert w4.w4a16_device_status() == 0
    for _, want, _, outs, _ in chains:
        for y in outs:
            assert torch.equal(y, want)


def _older(M, N, K):
    """A step of the kernels that begin before the one before them has ended: products of 16-bit
    activations (tensor pipe, prepared weights, FP4 weights) and a prompt on the 4-bit cache."""
    g = torch.Generator(device=DEV).manual_seed(M)
    w = torch.randn(N, K, device=DEV, generator=g)
    codes, scales, mins = w4.w4a16_quantize(w)
    qw = w4.w4a16_pack(codes)
    prep = w4.w4a16_prepare(qw, scales, mins)
    c4, s4, S = w4.nvfp4_quantize(w)
    x, few = (torch.randn(m, K, device=DEV, generator=g).bfloat16() for m in (M, 9))
    heads, kv_heads, dim = 8, 2, 128
    pages = (M + 63) // 64
    cache = w4.kv4_cache(pages, kv_heads, dim)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([M], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    q, k, v = (torch.randn(M, h, dim, device=DEV, generator=g).bfloat16()
               for h in (heads, kv_heads, kv_heads))
    w4.kv4_append(cache, table, lens, starts, k, v)

    def step():
        return [w4.w4a16_matmul(x, qw, scales, mins),
                w4.w4a16_matmul_prepared(x, qw, scales, mins, prep),
                w4.kv4_attention(q, cache, table, lens, starts, M, M),
                w4.nvfp4_matmul(few, c4, s4, S), w4.w4a16_matmul_prepared(few, qw, scales, mins, prep)]
    return step


@pytest.mark.parametrize("calls", [
    [("nvfp4", 300, 4096, 1024, 2), ("mxfp8", 16, 4096, 4096, 1)],
    [("mxfp4", 256, 2048, 4096, 4), ("nvfp4", 33, 2048, 8192, 1), ("mxfp8", 500, 2048, 4096, 3)]])
def test_beside_chains_of_kernels_that_begin_early(calls):
    chains = []
    for step in [_chain(*c) for c in calls] + [_older(300, 4096, 4096), _older(1000, 2048, 1024)]:
        want = step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [step() for _ in range(10)]
        chains.append((want, graph, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(100):
        for _, graph, _, stream in chains:
            with torch.cuda.stream(stream):
                graph.replay()
    ends = []
    for *_, stream in chains:
        ends.append(torch.cuda.Event())
        ends[-1].record(stream)
    until = time.monotonic() + 60
    while not all(e.query() for e in ends):
        assert time.monotonic() < until, "the chains stand still"
        time.sleep(0.001)
    assert w4.w4a16_device_status() == 0
    for want, _, outs, _ in chains:
        for y in outs:
            for a, b in zip(*((t if isinstance(t, list) else [t]) for t in (y, want))):
                assert torch.equal(a, b)
