"""Attention over the 4-bit key/value cache on the GPU: how near it is, and what no value, page or
buffer may do to it. Against sums in 64 bits of the values that the cache holds.

Bounds, from the arithmetic (a token's dim stands for c s + m, c a code of 0..15; "most" of it is
15 s + |m|; of a row, L = |scale| times the largest sum over the dims of |q| most of a visible key):
  * logits. A few rows: codes are FP16 subnormals 2^-22 c under an exponent of 2^-14, so a product's
    sum loses up to 2^-24 of 2^-14 |q| a step, 2^-16 |q| in units of codes, over at most 2 D / 16
    steps: 2^-12 |scale| max|q| s. Many rows: images exact or to 2^-22 of themselves. The rest is
    fp32, at most sixteen roundings or truncations to 2^-24 of L. E = 2^-12 |scale| max|q| max s +
    2^-20 L covers both;
  * lse: E, and 2^-17 for the fp32 sum of exponentials that are within 2^-21 of themselves, and its
    own rounding, 2^-22 |lse|;
  * a weight: each probability by a factor within e^(+-2E), and 2^-16 of itself for exponentials
    and sums; the sum with what was there before is rounded once, 2^-23 of it;
  * out: 2^-8.9 |out| + 2^-10 reach, reach = sum p most, and (e^2E - 1) reach. Rounding to BF16 takes
    up to 2^-8 |out|; where reach is twice |out| or more, as in sums of many values, the terms
    leave 2^-11 reach and more for the FP16 roundings of probabilities (times scales) and images,
    2^-11 each of a token's part and of either sign. So this is a bound on the kernels as they
    are, not one that every correct rounding keeps: a row of one value has its own (`sharp`)."""
import numpy as np
import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemv_w4a16_group_gb300") if torch.cuda.is_available() else None
DEV = "cuda"
FORMS = [(128, 64, 64), (128, 128, 16), (128, 32, 256), (64, 64, 16), (64, 32, 128)]


def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _bf16(x):
    return _gpu(np.asarray(x, np.float32)).bfloat16()


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def _held(x, group):
    """(x_hat, most, largest scale a token), fp64, of fp32 [n, H, D]."""
    q, s, m = ref.quantize(x, group)
    most = np.repeat(15.0 * s.astype(np.float64) + np.abs(m.astype(np.float64)), group, axis=-1)
    return ref.dequantize(q, s, m, group), most, s.astype(np.float64).max(-1)


class Batch:
    """Sequences whose keys and values are given as fp32 lists of [n, H, D], in a cache filled by
    kv4_append (equal bit for bit to the reference's, as other tests check)."""

    def __init__(self, ks, vs, group, page, seed=0):
        ks, vs = [ref.bf16(k) for k in ks], [ref.bf16(v) for v in vs]
        self.lens, self.group, self.page = [len(k) for k in ks], group, page
        _, self.H, self.D = ks[0].shape
        self.k, self.v = [_held(k, group) for k in ks], [_held(v, group) for v in vs]
        need = [(n + page - 1) // page for n in self.lens]
        order = np.random.default_rng(seed).permutation(sum(need) + 2).astype(np.int32)
        self.table = np.full((len(ks), max(need) + 1), -1, np.int32)
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.pages = len(order)
        # stale bytes are NaN parameters
        self.cache = torch.full((self.pages, self.H, page // 16, ref.record_bytes(self.D, group)),
                                0xFF, dtype=torch.uint8, device=DEV)
        w4.kv4_append(self.cache, _gpu(self.table), self.lens_t(), _gpu(_starts(self.lens)),
                      _bf16(np.concatenate(ks)), _bf16(np.concatenate(vs)), group=group)
        assert w4.w4a16_device_status() == 0

    def lens_t(self):
        return _gpu(np.array(self.lens, np.int32))


def _check(batch, q, new, scale=None, weights=True, table=None, gone=None, rows=None, status=0,
           copies=1, sharp=None):
    """Runs the attention of q (fp32 [T, heads, D]) and holds it to the bounds. gone[b]: positions
    that the call leaves out; rows: which of the T rows to look at; copies: the batch that many
    times over in one call, on the same pages, so that a CTA's share is long; sharp: rows whose
    logits lie so far apart that one token has all of the probability, whatever E (their out is one
    value to BF16, 2^-8 of itself, from an image of three roundings to FP16, 2^-9 most)."""
    q = ref.bf16(q)
    T, heads, D = q.shape
    H, G = batch.H, heads // batch.H
    scale = D ** -0.5 if scale is None else scale
    starts = _starts(new)
    table = batch.table if table is None else table
    width = table.shape[1] * batch.page
    before = np.random.default_rng(1).random((len(new), H, width)).astype(np.float32)
    lse_t = torch.full((copies * T, heads), 9.0, device=DEV)
    out_t = torch.full((copies * T, heads, D), 9.0, dtype=torch.bfloat16, device=DEV)
    w_t = torch.full((copies * len(new), H, width), 7.0, device=DEV) if weights else None
    w4.kv4_attention(_bf16(np.tile(q, (copies, 1, 1))), batch.cache,
                     _gpu(np.tile(table, (copies, 1))), batch.lens_t().repeat(copies),
                     _gpu(_starts(list(new) * copies)), max(max(batch.lens), 1), max(new),
                     group=batch.group, scale=scale, lse=lse_t, out=out_t,
                     weights=_gpu(np.tile(before, (copies, 1, 1))) if weights else None,
                     weights_out=w_t)
    assert w4.w4a16_device_status() == status

    def each(t):  # the copies first
        return t.double().cpu().numpy().reshape(copies, t.shape[0] // copies, *t.shape[1:])

    got, lse_g = each(out_t), each(lse_t)
    w_g = each(w_t) if weights else None
    look = np.ones(T, bool) if rows is None else rows
    for b, n in enumerate(batch.lens):
        mine = slice(starts[b], starts[b + 1])
        m = new[b]
        hide = np.arange(n) > np.arange(n - m, n)[:, None]
        if gone is not None:
            hide[:, gone[b]] = True
        w, w_tol = np.zeros((H, n)), np.zeros((H, n))
        for h in range(heads):
            g = h // G
            k, k_most, k_s = (x[:, g] for x in batch.k[b])
            v, v_most, _ = (x[:, g] for x in batch.v[b])
            x = q[mine, h].astype(np.float64)
            s = np.where(hide, -np.inf, scale * (x @ k.T))
            some = ~hide.all(1) if n else np.zeros(m, bool)
            top = s.max(1, keepdims=True, initial=-np.inf)
            top[~some] = 0
            e = np.exp(s - top)
            total = e.sum(1, keepdims=True)
            total[~some] = 1
            p, lse = e / total, (top + np.log(total))[:, 0]
            if m and n:
                L = abs(scale) * np.where(hide, 0, np.abs(x) @ k_most.T).max(1)
                E = (2.0 ** -12 * abs(scale) * np.abs(x).max(1)
                     * np.where(hide, 0, k_s[None]).max(1) + 2.0 ** -20 * L)
            else:
                E = np.zeros(m)
            grow = np.expm1(2 * (E if sharp is None else np.where(sharp[mine], 0, E)))
            want, reach = p @ v, p @ v_most
            ok = look[mine]
            tol = 2.0 ** -8.9 * np.abs(want) + (2.0 ** -10 + grow)[:, None] * reach
            if sharp is not None:
                one = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * reach
                tol = np.where(sharp[mine][:, None], one, tol)
            here, z = got[:, mine, h], lse_g[:, mine, h]
            assert np.isfinite(here[:, ok]).all()
            over = (np.abs(here - want) - tol)[:, ok]
            assert (over <= 0).all(), (b, h, over.max(), np.abs(want).max())
            assert np.isneginf(z[:, ~some]).all() and (here[:, ~some] == 0).all()
            over = (np.abs(z - lse) - (E + 2.0 ** -17 + 2.0 ** -22 * np.abs(lse)))[:, some & ok]
            assert (over <= 0).all(), (b, h, over.max())
            w[g] += p[some].sum(0)
            w_tol[g] += ((grow + 2.0 ** -16)[:, None] * p)[some].sum(0)
        if weights:
            old = before[b].astype(np.float64)
            assert (w_g[:, b, :, n:] == 7.0).all()
            if rows is None:
                d = np.abs(w_g[:, b, :, :n] - old[:, :n] - w)
                assert (d <= w_tol + 2.0 ** -23 * (old[:, :n] + w)).all(), d.max()


def _normal(g, n, H, D, wide=True):
    chan = np.where(g.random((H, D)) < 0.05, 4.0, 1.0) if wide else 1.0
    return g.standard_normal((n, H, D)) * chan, g.standard_normal((n, H, D))


def _random(lens, H, D, group, page, seed):
    g = np.random.default_rng(seed)
    kv = [_normal(g, n, H, D) for n in lens]
    return Batch([k for k, _ in kv], [v for _, v in kv], group, page, seed), g


# ---- nearness, with and without weights ---------------------------------------------------
@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("heads,H,lens,new", [
    (4, 1, [1], [1]), (4, 2, [17, 1, 64, 129], [1, 1, 1, 1]), (12, 2, [900, 3], [1, 1]),
    (4, 1, [700, 40], [5, 8]), (8, 4, [333, 1000], [4, 1]), (3, 1, [90, 2], [30, 2]),
    (4, 1, [150, 60], [150, 1]), (6, 2, [700, 257, 5], [300, 257, 5])])
def test_out_lse_and_weights(D, group, page, weights, heads, H, lens, new):
    batch, g = _random(lens, H, D, group, page, 40)
    _check(batch, g.standard_normal((sum(new), heads, D)), new, weights=weights)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("new", [1, 9, 130])
def test_a_long_sequence(weights, new):
    batch, g = _random([9000], 2, 128, 64, 64, 41)
    _check(batch, g.standard_normal((new, 8, 128)), [new], weights=weights)


# ---- values of one size in a group --------------------------------------------------------
def _rising(n, H, D, a_unit, seed):
    """Keys whose logits under q near 1 rise by a_unit (base 2) in 32 tokens."""
    step = a_unit / 32 / (D ** 0.5 * 1.4426950408889634)
    g = np.random.default_rng(seed)
    return np.arange(n)[:, None, None] * step + 1e-3 * g.standard_normal((n, H, D)), g


@pytest.mark.parametrize("D,group,value", [(128, 64, 0.0), (128, 128, 1.0), (64, 32, 1.0),
                                           (64, 64, 0.0), (128, 32, -3e-38)])
@pytest.mark.parametrize("a_unit", [0.2, 0.6, 1.1])
@pytest.mark.parametrize("heads", [4, 8, 16])
def test_constant_values(D, group, value, a_unit, heads):
    """Scales of 0 and logits that rise from unit to unit, in a batch that gives every warp several
    units of a segment."""
    n, B, H = 2048, 32, 2
    k, g = _rising(n, H, D, a_unit, 42)
    batch = Batch([k], [np.full((n, H, D), value)], group, 64)
    q = 1 + 0.02 * g.standard_normal((1, heads, D))
    # every sequence of the batch reads the same pages
    table = _gpu(np.repeat(batch.table, B, 0))
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out = w4.kv4_attention(_bf16(np.repeat(q, B, 0)), batch.cache, table, lens,
                           _gpu(_starts([1] * B)), n, 1, group=group).float()
    assert w4.w4a16_device_status() == 0
    want = torch.tensor(value).bfloat16().item()
    # probabilities sum to 1 within 2^-17 and the BF16 value is rounded to again
    assert torch.isfinite(out).all()
    assert ((out - want).abs() <= 2.0 ** -8 * abs(want)).all()


# ---- values of any size -------------------------------------------------------------------
# (heads on two, new tokens, copies): a call that is cut to the last unit, and one whose CTAs go
# through whole sequences
PATHS = [(8, 1, 1), (8, 1, 60), (8, 4, 60), (4, 30, 60), (4, 130, 1), (4, 130, 60)]


@pytest.mark.parametrize("heads,new,copies", PATHS)
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("size", [1e-30, 1e-3, 1e-2, 1e30, 1e35])
def test_values_of_one_size(heads, new, copies, D, group, size):
    g = np.random.default_rng(43)
    k, v = _normal(g, 900, 2, D)
    _check(Batch([k], [v * size], group, 64), g.standard_normal((new, heads, D)), [new],
           copies=copies)


@pytest.mark.parametrize("heads,new,copies", PATHS)
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3])
@pytest.mark.parametrize("zeros", [[(0, 128)], [(256, 512)], [(0, 128), (300, 301), (640, 768)]])
def test_tiles_of_zeros(heads, new, copies, D, group, size, zeros):
    g = np.random.default_rng(44)
    k, v = _normal(g, 900, 2, D)
    v *= size
    for lo, hi in zeros:
        v[lo:hi] = 0
    _check(Batch([k], [v], group, 64), g.standard_normal((new, heads, D)), [new], copies=copies)


def _with_unlikely(g, n, D, at, size, far):
    """Keys under which the tokens `at` have logits `far` nats below the others', and values that
    are `size` times the others' there. Queries are near 1 in half of the dims."""
    k, v = _normal(g, n, 2, D, wide=False)
    k[at] = -far / (D ** 0.5 / 2) + 0.1 * k[at]
    k[..., D // 2:] = 0.5 * g.standard_normal((n, 2, D // 2))
    v[at] *= size
    return k, v


def _near_one(g, new, heads, D):
    q = 1 + 0.05 * g.standard_normal((new, heads, D))
    q[..., D // 2:] = 0.3 * g.standard_normal((new, heads, D // 2))
    return q


@pytest.mark.parametrize("heads,new,copies", PATHS)
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("at", [[3], [400], [5, 600]])
@pytest.mark.parametrize("power", [14, 20, 30])
def test_a_large_value_that_is_hardly_attended(heads, new, copies, D, group, at, power):
    """A token whose values are 2^power times the others' and whose probability is e^-60 or less
    takes no bits from the others'."""
    g = np.random.default_rng(45)
    k, v = _with_unlikely(g, 900, D, at, 2.0 ** power, 60.0)
    _check(Batch([k], [v], group, 64), _near_one(g, new, heads, D), [new], copies=copies)


@pytest.mark.parametrize("heads,new,copies", PATHS)
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
def test_a_first_token_with_most_of_the_weight_and_small_values(heads, new, copies, D, group):
    g = np.random.default_rng(46)
    k, v = _normal(g, 900, 2, D, wide=False)
    k[0] = 0.8 + 0.1 * k[0]
    v[0] *= 2.0 ** -10
    _check(Batch([k], [v], group, 64), 1 + 0.3 * g.standard_normal((new, heads, D)), [new],
           copies=copies)


@pytest.mark.parametrize("heads,new", [(4, 130), (8, 200), (2, 4), (4, 24)])
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("size", [1e5, 1e15, 1e30])
def test_hidden_tokens_of_any_size(heads, new, D, group, size):
    """The last tokens hold huge finite keys and values: rows that do not see them are as near as
    without them."""
    g = np.random.default_rng(47)
    n, last = 600, 3
    k, v = _normal(g, n, 2, D)
    k[n - last:] *= size
    v[n - last:] *= size
    rows = np.arange(new) < new - last
    _check(Batch([k], [v], group, 64), g.standard_normal((new, heads, D)), [new], rows=rows)


def _sharp(batch, q, new, big, power):
    """Which rows of `big` (one sequence, queries of 2^power) have a best logit ahead of the next by
    far more than its error, 2^-20 L, L about 50 2^power, in all heads."""
    heads, D = q.shape[1:]
    x, n = ref.bf16(q).astype(np.float64), batch.lens[0]
    big = big.copy()
    for h in range(heads):
        k = batch.k[0][0][:, h // (heads // batch.H)]
        for i in np.flatnonzero(big):
            s = np.sort(D ** -0.5 * x[i, h] @ k[:n - new + i + 1].T)
            big[i] &= s[-1] - s[-2] > 2.0 ** (power - 10)
    return big


@pytest.mark.parametrize("heads,new", [(4, 130), (8, 300), (8, 4), (4, 24)])
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("power", [14, 24, 40])
def test_logits_of_any_size(heads, new, D, group, power):
    """Logits far beyond what exponentials of a difference rounded once would bear: a row is the
    token of its largest logit."""
    g = np.random.default_rng(54)
    n = 600
    k, v = _normal(g, n, 2, D)
    q = g.standard_normal((new, heads, D)) * 2.0 ** power
    batch = Batch([k], [v], group, 64)
    big = _sharp(batch, q, new, np.ones(new, bool), power)
    assert big.mean() > 0.8
    _check(batch, q, [new], rows=None if big.all() else big, sharp=big)


@pytest.mark.parametrize("heads,new", [(4, 130), (8, 300), (8, 4), (4, 24)])
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("power", [14, 24, 40])
@pytest.mark.parametrize("at", [0, 7])
def test_rows_of_any_size(heads, new, D, group, power, at):
    """Queries of every eighth token are 2^power times the others': each row as near as without
    them. Theirs see one token alone."""
    g = np.random.default_rng(53)
    n = 600
    k, v = _normal(g, n, 2, D)
    large = np.arange(new) % 8 == at
    q = g.standard_normal((new, heads, D))
    q[large] *= 2.0 ** power
    batch = Batch([k], [v], group, 64)
    big = _sharp(batch, q, new, large, power)
    rows = big | ~large
    assert rows.mean() > 0.9
    _check(batch, q, [new], rows=None if rows.all() else rows, sharp=big)


# ---- pages that are not there -------------------------------------------------------------
@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("heads,new", [(4, [1, 1]), (4, [3, 1]), (8, [9, 2]), (4, [130, 1]),
                                       (4, [90, 65])])
@pytest.mark.parametrize("weights", [False, True])
def test_tokens_of_a_missing_page_are_left_out(D, group, page, heads, new, weights):
    lens = [700, 300]
    batch, g = _random(lens, 2, D, group, page, 48)
    table = batch.table.copy()
    gone = [np.zeros(n, bool) for n in lens]
    for b, at, bad in ((0, 1, -1), (0, 500 // page, 1 << 30), (1, 0, batch.pages)):
        table[b, at] = bad
        gone[b][at * page:(at + 1) * page] = True
    q = g.standard_normal((sum(new), heads, D))
    _check(batch, q, new, weights=weights, table=table, gone=gone, status=8)
    _check(batch, q, new, weights=weights)


@pytest.mark.parametrize("new", [1, 40, 130])
def test_a_sequence_without_any_page(new):
    lens = [300, 200]
    batch, g = _random(lens, 2, 128, 64, 64, 49)
    table = batch.table.copy()
    table[1] = -1
    gone = [np.zeros(300, bool), np.ones(200, bool)]
    _check(batch, g.standard_normal((2 * new, 4, 128)), [new, new], table=table, gone=gone, status=8)


@pytest.mark.parametrize("D,group,page", FORMS[:4])
def test_eviction_leaves_a_missing_page_where_it_is(D, group, page):
    """The same tokens are kept; those of the page are not moved, and their places stay as they
    were."""
    n, budget, H = 520, 300, 2
    batch, g = _random([n], H, D, group, page, 51)
    fill = batch.pages
    width = (budget + page - 1) // page
    spare = torch.full((width,) + batch.cache.shape[1:], 0x3A, dtype=torch.uint8, device=DEV)
    out_table = np.arange(fill, fill + width, dtype=np.int32)[None]
    table = batch.table.copy()
    table[0, 1] = -1
    w = _gpu(g.random((1, H, n)).astype(np.float32))
    res = []
    for t, status in ((batch.table, 0), (table, 8)):
        cache = torch.cat([batch.cache, spare])
        kept, lens, _ = w4.kv4_evict(cache, _gpu(t), batch.lens_t(), w, _gpu(out_table), budget, n,
                                     D, first=2, recent=20, group=group)
        assert w4.w4a16_device_status() == status and lens.item() == budget
        res.append((kept.cpu().numpy(), ref.Cache(cache.cpu().numpy(), out_table, D, group)))
    before = ref.Cache(torch.cat([batch.cache, spare]).cpu().numpy(), out_table, D, group)
    assert np.array_equal(res[0][0], res[1][0])
    assert torch.equal(torch.from_numpy(res[1][1].data[:fill]), batch.cache.cpu())
    for h in range(H):
        gone = res[0][0][0, h] // page == 1
        assert gone.any() and not gone.all()
        for x, moved, old in zip(*(c.get(0, h, budget) for c in (res[1][1], res[0][1], before))):
            assert np.array_equal(x, np.where(gone[:, None], old, moved))


# ---- streams ------------------------------------------------------------------------------
def test_a_raw_stream_handle():
    """A call on a raw handle runs on that stream alone, its scratch and results included: nothing
    of it waits for the current stream, which is kept busy meanwhile."""
    batch, g = _random([3000, 700], 2, 128, 64, 64, 52)
    table, lens = _gpu(batch.table), batch.lens_t()
    spare = torch.zeros((8,) + batch.cache.shape[1:], dtype=torch.uint8, device=DEV)
    cache = torch.cat([batch.cache, spare])
    out_table = _gpu(np.arange(8, dtype=np.int32).reshape(2, 4) + batch.pages)
    weights = _gpu(g.random((2, 2, 3000)).astype(np.float32))
    calls = []
    for new in (1, 30, 90):
        starts = _gpu(_starts([new, new]))
        q = _bf16(g.standard_normal((2 * new, 8, 128)))
        calls.append(lambda s, q=q, new=new, starts=starts: [w4.kv4_attention(
            q, cache, table, lens, starts, 3000, new, stream=s)])
    starts = _gpu(_starts([300, 90]))
    calls.append(lambda s: w4.kv4_read(cache, table, lens, starts, 390, 128, stream=s))
    calls.append(lambda s: w4.kv4_evict(cache, table, lens, weights, out_table, 200, 3000, 128,
                                        first=1, recent=9, stream=s))
    want = [call(None) for call in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for call in calls:  # allocations that wait for the device are behind us
        call(side.cuda_stream)
    side.synchronize()
    torch.cuda._sleep(400_000_000)
    busy = torch.cuda.Event()
    busy.record()
    got = [call(side.cuda_stream) for call in calls]
    side.synchronize()
    assert not busy.query()
    got = [[t.cpu() for t in r] for r in got]
    for a, b in zip(want, got):
        assert all(torch.equal(x.cpu(), y) for x, y in zip(a, b))
    for handle in (0, torch.cuda.default_stream().cuda_stream):
        assert torch.equal(calls[0](handle)[0], want[0][0])
    assert w4.w4a16_device_status() == 0


# ---- one workspace for calls of any shape -------------------------------------------------
def test_one_workspace_for_calls_of_any_shape():
    """Larger and smaller batches, few rows and prompts, with weights and without: each call gives
    what it gives with a workspace of its own."""
    D, H, group = 128, 2, 64
    shapes = [([3000], [1], 4), ([3000] * 40, [1] * 40, 4), ([2000] * 48, [2] * 48, 12),
              ([3000], [300], 4), ([2000] * 48, [2] * 48, 12), ([3000, 700, 90], [1, 5, 3], 8),
              ([3000, 2000], [150, 1], 4), ([500] * 90, [3] * 90, 6), ([3000], [1], 4)]
    batch, g = _random([3000], H, D, group, 64, 50)

    def size(lens, new, heads, weights):
        return w4.kv4_attention_workspace_bytes(len(lens), sum(new), max(new), max(lens), heads, H,
                                                D, group, weights)

    shared = torch.zeros(max(size(*s, True) for s in shapes), dtype=torch.uint8, device=DEV)
    for weights in (True, False, True):
        for lens, new, heads in shapes:
            q = _bf16(g.standard_normal((sum(new), heads, D)))
            args = (q, batch.cache, _gpu(np.repeat(batch.table, len(lens), 0)),
                    _gpu(np.array(lens, np.int32)), _gpu(_starts(new)), max(lens), max(new))
            res = []
            for ws in (shared, torch.zeros(size(lens, new, heads, weights), dtype=torch.uint8,
                                           device=DEV)):
                out = torch.full_like(q, 9.0)
                w = torch.full((len(lens), H, max(lens)), 9.0, device=DEV) if weights else None
                w4.kv4_attention(*args, group=group, out=out, weights_out=w, workspace=ws)
                res.append((out, w))
            assert torch.equal(res[0][0], res[1][0])
            assert not weights or torch.equal(res[0][1], res[1][1])
    assert w4.w4a16_device_status() == 0
