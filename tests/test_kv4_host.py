"""The 4-bit key/value cache without a GPU: sizes, refusals before any launch, and the
reference's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_reference as ref

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 6
A, B = 0x10000, 0x20000  # never dereferenced


class Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p)]
    _fields_ += [(n, ctypes.c_int32) for n in ("pages", "kv_heads", "head_dim", "group",
                                               "page_size", "batch", "table_width")]


GOOD = dict(data=A, table=A + 4, lens=A + 4, pages=10, kv_heads=2, head_dim=128, group=64,
            page_size=16, batch=2, table_width=4)


@pytest.fixture(scope="module")
def lib(cuda_lib):
    lib = ctypes.CDLL(cuda_lib)
    P, I, L, S, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                     ctypes.c_float)
    C = ctypes.POINTER(Cache)
    lib.kv4_append.argtypes = [C, P, P, L, P, L, I, P, I, P]
    lib.kv4_read.argtypes = [C, P, P, P, I, P]
    lib.kv4_attention.argtypes = [C, P, P, L, P, P, I, I, I, I, F, P, P, I, P, S, P]
    lib.kv4_evict.argtypes = [C, P, I, P, I, I, I, I, I, P, P, P, I, P]
    lib.kv4_cache_bytes.restype = S
    lib.kv4_attention_workspace_bytes.restype = S
    lib.w4a16_status_string.restype = ctypes.c_char_p
    return lib


def _append(lib, cache, starts=A, k=A, ks=256, v=A, vs=256, tokens=3, w=None, wl=0):
    return lib.kv4_append(cache, starts, k, ks, v, vs, tokens, w, wl, None)


def _read(lib, cache, starts=A, k=A, v=A, tokens=3):
    return lib.kv4_read(cache, starts, k, v, tokens, None)


def _attention(lib, cache, starts=A, q=A, qs=512, out=B, lse=None, tokens=3, heads=4, max_new=2,
               max_len=64, scale=0.1, w=None, wo=None, wl=0, ws=A, wsb=1 << 40):
    return lib.kv4_attention(cache, starts, q, qs, out, lse, tokens, heads, max_new, max_len,
                             scale, w, wo, wl, ws, wsb, None)


def _evict(lib, cache, ot=A, ow=2, w=A, wl=64, budget=20, first=1, recent=3, max_len=64, kept=A,
           nl=B, wo=B, wol=20):
    return lib.kv4_evict(cache, ot, ow, w, wl, budget, first, recent, max_len, kept, nl, wo, wol,
                         None)


CALLS = [_append, _read, _attention, _evict]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("change,status", [
    (dict(data=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(pages=0), INVALID), (dict(kv_heads=0), INVALID), (dict(batch=-1), INVALID),
    (dict(table_width=0), INVALID), (dict(page_size=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(group=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(group=16), UNSUPPORTED), (dict(head_dim=64, group=128), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=1 << 20, table_width=1 << 11), UNSUPPORTED),
    (dict(data=A + 8), MISALIGNED), (dict(lens=A + 2), MISALIGNED), (dict(table=A + 1), MISALIGNED)])
def test_every_call_checks_the_cache(lib, call, change, status):
    assert call(lib, Cache(**{**GOOD, **change})) == status


@pytest.mark.parametrize("call", CALLS)
def test_null_cache(lib, call):
    assert call(lib, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(starts=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(tokens=0), INVALID), (dict(ks=255), INVALID), (dict(ks=260), INVALID),
    (dict(vs=248), INVALID), (dict(w=A, wl=63), INVALID), (dict(k=A + 8), MISALIGNED),
    (dict(v=A + 2), MISALIGNED), (dict(starts=A + 2), MISALIGNED),
    (dict(w=A + 2, wl=64), MISALIGNED)])
def test_append_refusals(lib, change, status):
    assert _append(lib, Cache(**GOOD), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(starts=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(tokens=-1), INVALID), (dict(k=A + 8), MISALIGNED), (dict(v=A + 8), MISALIGNED)])
def test_read_refusals(lib, change, status):
    assert _read(lib, Cache(**GOOD), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(starts=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(tokens=0), INVALID), (dict(heads=0), INVALID), (dict(heads=3), INVALID),
    (dict(max_new=0), INVALID), (dict(max_new=4), INVALID), (dict(max_len=0), INVALID),
    (dict(max_len=65), INVALID), (dict(qs=504), INVALID), (dict(qs=516), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(w=A), INVALID), (dict(wo=A, wl=63), INVALID), (dict(q=A + 8), MISALIGNED),
    (dict(out=A + 4), MISALIGNED), (dict(lse=A + 2), MISALIGNED), (dict(ws=A + 8), MISALIGNED),
    (dict(wo=A + 1, wl=64), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE)])
def test_attention_refusals(lib, change, status):
    assert _attention(lib, Cache(**GOOD), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(ot=None), INVALID), (dict(w=None), INVALID), (dict(kept=None), INVALID),
    (dict(nl=None), INVALID), (dict(wo=None), INVALID), (dict(ow=0), INVALID),
    (dict(budget=0), INVALID), (dict(first=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(first=10, recent=11), INVALID), (dict(wl=63), INVALID), (dict(wol=19), INVALID),
    (dict(max_len=65), INVALID), (dict(budget=33, wol=33), INVALID), (dict(w=A, wo=A), INVALID),
    (dict(nl=A + 4), INVALID), (dict(kept=A + 2), MISALIGNED), (dict(ot=A + 3), MISALIGNED)])
def test_evict_refusals(lib, change, status):
    assert _evict(lib, Cache(**GOOD), **change) == status


def test_sizes(lib):
    assert lib.kv4_cache_bytes(10, 8, 128, 64, 64) == 10 * 8 * 64 * 144   # 4.5 bits a value
    assert lib.kv4_cache_bytes(1, 1, 128, 128, 16) == 16 * 136            # 4.25 bits
    assert lib.kv4_cache_bytes(1, 1, 64, 32, 16) == 16 * 80
    for bad in ((0, 1, 128, 64, 16), (1, 1, 100, 64, 16), (1, 1, 128, 48, 16), (1, 1, 128, 64, 24)):
        assert lib.kv4_cache_bytes(*bad) == 0
    ws = lib.kv4_attention_workspace_bytes
    assert ws(1, 1, 1, 100, 5, 2, 128, 64, 0) == 0                        # heads % kv_heads
    assert ws(1, 1, 1, 100, 4, 2, 96, 64, 0) == 0
    assert lib.w4a16_status_string(8) == b"W4A16_ERR_INDEX"


def test_reference_quantizer_by_hand():
    x = np.linspace(0, 15, 32, dtype=np.float32)
    q, s, m = ref.quantize(ref.bf16(x)[None], 32)
    assert s[0, 0] == 1 and m[0, 0] == 0 and q[0, 0] == 0 and q[0, -1] == 15
    q, s, m = ref.quantize(np.full((1, 32), 2.5, np.float32), 32)
    assert s[0, 0] == 0 and m[0, 0] == 2.5 and not q.any()
    # ties go to the even code: (x - m) / s = 0.5, 1.5, 2.5
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [15, 0.5, 1.5, 2.5]
    q, _, _ = ref.quantize(x, 32)
    assert q[0, :4].tolist() == [15, 0, 2, 2]


@pytest.mark.parametrize("D,group", [(128, 64), (128, 128), (128, 32), (64, 32), (64, 64)])
def test_reference_layout_round_trip(D, group):
    g = np.random.default_rng(0)
    n, H = 37, 2
    cache = ref.Cache(np.zeros((3, H, 1, ref.record_bytes(D, group)), np.uint8),
                      np.array([[2, 0, 1]], np.int32), D, group)
    k, v = ref.bf16(g.standard_normal((n, H, D))), ref.bf16(g.standard_normal((n, H, D)))
    kk, vv = ref.quantize(k, group), ref.quantize(v, group)
    for p in range(n):
        for h in range(H):
            cache.put(0, h, p, *(x[p, h] for x in kk), *(x[p, h] for x in vv))
    for h in range(H):
        k2, v2 = cache.get(0, h, n)
        assert np.array_equal(k2, ref.dequantize(*kk, group)[:, h])
        assert np.array_equal(v2, ref.dequantize(*vv, group)[:, h])
        step = np.repeat(kk[1][:, h], group, axis=1)
        assert (np.abs(k2 - k[:, h]) <= 0.51 * step + 2.0 ** -7 * np.abs(k[:, h])
                + 0.05 * step).all()


def test_reference_layout_words():
    """One code at a time, where the description puts it."""
    D, group = 128, 64
    rec = ref.record_bytes(D, group)
    for t, d, kw, kbit, vw, vbit in [(0, 0, 0, 0, 0, 0), (0, 1, 0, 16, 0, 4), (0, 8, 4, 0, 8, 0),
                                     (1, 34, 17, 4, 1, 24), (15, 127, 255, 28, 255, 28)]:
        cache = ref.Cache(np.zeros((1, 1, 1, rec), np.uint8), np.zeros((1, 1), np.int32), D, group)
        k = np.zeros(D, int)
        k[d] = 9
        z = np.zeros(2, np.float32)
        cache.put(0, 0, t, k, z, z, k, z, z)
        w = cache.data[0, 0, 0].view(np.uint32)
        v0 = (8 * D + 64 * 2) // 4
        assert w[kw] == 9 << kbit and w[v0 + vw] == 9 << vbit and np.count_nonzero(w) == 2


@pytest.mark.parametrize("stream,on", [(None, None), (0, "default"), (1, "default"),
                                       (0x5550, 0x5550)])
@pytest.mark.parametrize("zero", [False, True])
def test_memory_of_a_call_is_its_streams(cuda_lib, monkeypatch, stream, on, zero):
    """Scratch and results of a call on a raw handle are allocated, and filled, under it."""
    import contextlib

    import gemv_w4a16_group_gb300 as w4

    under, seen = [None], []

    @contextlib.contextmanager
    def enter(s):
        under.append(s)
        yield
        under.pop()

    def empty(*args, real=torch.empty, **kw):
        seen.append(under[-1])
        return real(*args, **kw)

    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch, "empty", empty)
    t = w4._new(torch.zeros(1), (5,), torch.uint8, stream, zero=zero)
    assert seen == [on] and t.shape == (5,) and (not zero or not t.any())
