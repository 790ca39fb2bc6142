"""The 4-bit key/value cache in plain numpy, 64-bit sums, for the tests (no GPU).

Written from the format's description in include/w4a16.h, dim by dim; shares nothing with the
kernels."""
import numpy as np
import torch


def bf16(x):
    """Round to BF16, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()


def bf16_bits(x):
    return (np.ascontiguousarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint32)


def record_bytes(D, group):
    return 16 * (D + 8 * (D // group))


def quantize(x, group):
    """fp32 [..., D] (BF16 values) -> codes int [..., D], scales, minimums fp32 [..., D/group]."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    mn, mx = g.min(-1), g.max(-1)
    s = bf16((mx - mn) / np.float32(15))
    m = bf16(mn)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((g - m[..., None]) / s[..., None])   # half to even
    q = np.where(s[..., None] == 0, 0, np.clip(np.nan_to_num(q), 0, 15)).astype(np.uint32)
    return q.reshape(x.shape), s, m


def dequantize(q, s, m, group):
    return (q.astype(np.float64).reshape(*q.shape[:-1], q.shape[-1] // group, group) * s[..., None].astype(np.float64)
            + m[..., None].astype(np.float64)).reshape(q.shape)


class Cache:
    """uint8 [pages, heads, page / 16, record] with a page table."""

    def __init__(self, data, table, D, group):
        self.data, self.table, self.D, self.group = data, table, D, group
        self.page = data.shape[2] * 16

    def _at(self, b, h, pos):
        """Index of the records of positions pos, and the tokens' rows in them."""
        return (self.table[b, pos // self.page], h, pos % self.page // 16), pos % 16

    def put(self, b, h, pos, kq, ks, km, vq, vs, vm):
        """Codes [n, D] (or [D]), scales and minimums [n, D / group] of the tokens at pos."""
        D, NB, NG = self.D, self.D // 32, self.D // self.group
        pos = np.atleast_1d(np.asarray(pos))
        kq, vq = np.atleast_2d(kq).astype(np.uint32), np.atleast_2d(vq).astype(np.uint32)
        (page, _, rec), t = self._at(b, h, pos)
        words = self.data.view(np.uint32)
        v0 = (8 * D + 64 * NG) // 4

        # the dims of a token all go to different fields, so whole rows are set at once
        d = np.arange(D)
        for i in range(len(pos)):
            w = words[page[i], h, rec[i]]
            ti = t[i]
            for at, bit, code in (
                    (ti * 4 * NB + d % 32 // 8 * NB + d // 32, 4 * (d % 8 // 2) + 16 * (d % 2), kq[i]),
                    (v0 + (ti // 2 * 8 + d % 32 // 4) * NB + d // 32, 16 * (ti % 2) + 4 * (d % 4),
                     vq[i])):
                bit = bit.astype(np.uint32)
                np.bitwise_and.at(w, at, ~(np.uint32(15) << bit))
                np.bitwise_or.at(w, at, code << bit)
        ks, km, vs, vm = (np.atleast_2d(x) for x in (ks, km, vs, vm))
        for base, sc, mn in ((2 * D, ks, km), (v0 + 2 * D, vs, vm)):
            for g in range(NG):
                words[page, h, rec, base + 16 * g + t] = bf16_bits(sc[:, g]) | (
                    bf16_bits(mn[:, g]) << np.uint32(16))

    def get(self, b, h, n):
        """K, V fp64 [n, D] of the first n tokens."""
        D, NB, NG = self.D, self.D // 32, self.D // self.group
        pos, d = np.arange(n), np.arange(D)
        at, t = self._at(b, h, pos)
        w = self.data[at].view(np.uint32)           # a token's record
        i, t = pos[:, None], t[:, None]
        v0 = (8 * D + 64 * NG) // 4
        kc = (w[i, t * 4 * NB + d % 32 // 8 * NB + d // 32]
              >> (4 * (d % 8 // 2) + 16 * (d % 2)).astype(np.uint32)) & 15
        vc = (w[i, v0 + (t // 2 * 8 + d % 32 // 4) * NB + d // 32]
              >> (16 * (t % 2) + 4 * (d % 4)).astype(np.uint32)) & 15
        res = []
        for code, base in ((kc, 2 * D), (vc, v0 + 2 * D)):
            p = w[i, base + 16 * (d // self.group) + t]
            sc = (p << np.uint32(16)).view(np.float32).astype(np.float64)
            mn = (p & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
            with np.errstate(invalid="ignore"):
                res.append(code * sc + mn)
        return res


def attention(q, cache, lens, starts, heads, kv_heads, scale):
    """out, lse, weights [batch, kv_heads, max len], and the bound's terms: reach = sum p (|code
    scale| + |min|) as |v - min| + |min| is at most that, span = largest sum |q k| scale of a row."""
    T, G = q.shape[0], heads // kv_heads
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    reach, span = np.zeros(q.shape), np.zeros(q.shape[:2])
    weights = np.zeros((len(lens), kv_heads, max(max(lens), 1)))
    for b, n in enumerate(lens):
        m = starts[b + 1] - starts[b]
        for g in range(kv_heads):
            k, v = cache.get(b, g, n)
            lo = v.min(1, keepdims=True) if n else v[:, :1]
            terms = np.abs(v - lo) + np.abs(lo)
            for h in range(g * G, (g + 1) * G):
                rows = slice(starts[b], starts[b + 1])
                x = q[rows, h].astype(np.float64)
                hide = np.arange(n) > np.arange(n - m, n)[:, None]
                s = np.where(hide, -np.inf, scale * (x @ np.where(np.isfinite(k), k, 0.0).T))
                some = ~hide.all(1) if n else np.zeros(m, bool)
                if not some.any():
                    continue
                top = s[some].max(1, keepdims=True)
                z = top + np.log(np.exp(s[some] - top).sum(1, keepdims=True))
                p = np.zeros(s.shape)
                p[some] = np.exp(s[some] - z)
                out[rows, h] = p @ v
                reach[rows, h] = p @ terms
                lse[rows, h][some] = z[:, 0]
                weights[b, g, :n] += p.sum(0)
                reachable = np.where(hide, 0.0, np.abs(x) @ np.abs(k).T)
                span[rows, h] = abs(scale) * reachable.max(1)
    return out, lse, weights, reach, span


def evict(weights, lens, budget, first, recent):
    """kept int [batch, heads, budget] (-1 past the length)."""
    B, H, _ = weights.shape
    kept = np.full((B, H, budget), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(H):
            if n <= budget:
                kept[b, h, :n] = np.arange(n)
                continue
            w = weights[b, h, :n].astype(np.float64)
            w = np.where(np.isnan(w), -np.inf, w)
            mid = list(range(first, n - recent))
            mid.sort(key=lambda i: (-w[i], i))
            idx = list(range(first)) + mid[:budget - first - recent] + list(range(n - recent, n))
            kept[b, h] = sorted(idx)
    return kept
