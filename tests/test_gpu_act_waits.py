"""Products whose waits run out: whatever the limit, an element of y is the right one or as it was,
and the device's status says that a wait ran out where one is missing."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"
OK, TIMEOUT = 0, 5
BEFORE = 0x7FD3  # what y holds before a call, as bits: a NaN that no product gives
BLOCKS = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


@pytest.fixture
def settings():
    limit, kernel = w4.testing_set_act_wait_limit(0), w4.testing_set_act_kernel(-1)
    yield
    w4.testing_set_act_wait_limit(limit)
    w4.testing_set_act_kernel(kernel)


def _product(form, M, N, K):
    """A call that writes into a given y: codes from the whole range, block scales of 1."""
    g = torch.Generator(device=DEV).manual_seed(M + N)

    def codes(rows, width, keep):
        return torch.randint(0, 256, (rows, width), dtype=torch.uint8, device=DEV,
                             generator=g) & keep

    def tiles(rows):
        one = 0x38 if form == "nvfp4" else 127
        return torch.full(((rows + 127) // 128, K // BLOCKS[form] // 4, 512), one,
                          dtype=torch.uint8, device=DEV)

    w, sw, sx = codes(N, K // 2, 0xFF), tiles(N), tiles(M)
    if form == "nvfp4":
        x, rows, S = codes(M, K // 2, 0xFF), torch.ones(M, device=DEV), torch.ones(1, device=DEV)
        return lambda y: w4.nvfp4_matmul_act(x, sx, rows, w, sw, S, y=y)
    x = codes(M, K // 2, 0xFF) if form == "mxfp4" else codes(M, K, 0xB7)
    return lambda y: w4.mxfp4_matmul_act(x, sx, w, sw, y=y)


# Clusters of CTAs that send their parts, and that read one another's; single CTAs; pairs, alone
# with more than one tile each, and two and four that share one. A wait looks at the clock after a
# few hundred microseconds, so the rows are long.
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("kernel,M,N,K", [
    (1, 5, 520, 1 << 22), (1, 40, 264, 1 << 22), (1, 100, 130, 1 << 22), (1, 3, 40000, 1 << 16),
    (2, 2100, 2600, 1 << 18), (3, 300, 1032, 1 << 20), (4, 200, 520, 1 << 21)])
def test_expired_waits(settings, form, kernel, M, N, K):
    w4.testing_set_act_kernel(kernel)
    call = _product(form, M, N, K)

    def run(ns):
        w4.testing_set_act_wait_limit(ns)
        y = torch.full((M, N), BEFORE, dtype=torch.int16, device=DEV)
        torch.cuda.synchronize()
        began = time.perf_counter()
        call(y.view(torch.bfloat16))
        status = w4.w4a16_device_status()
        return y, status, time.perf_counter() - began

    run(10 ** 9)
    want, status, took = run(10 ** 9)
    assert status == OK and not (want == BEFORE).any()
    expired = 0
    for share in [0] + [0.025 * i for i in range(41)]:
        y, status, _ = run(max(1, int(share * took * 1e9)))
        kept = y == BEFORE
        assert status in (OK, TIMEOUT)
        assert torch.equal(torch.where(kept, want, y), want), f"limit {share} of the call"
        assert status == TIMEOUT or not kept.any()
        expired += status == TIMEOUT
    assert expired > 0 or K < 1 << 18  # (single CTAs' tiles are too short for the clock)
    y, status, _ = run(10 ** 9)
    assert status == OK and torch.equal(y, want)
