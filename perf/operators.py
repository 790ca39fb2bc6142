"""The 4-bit key/value cache: what is measured of its operators.

Four operators that a decoder on 4-bit weights needs beside its matrix products:

  * ``kv4_append``    quantizes the keys and values of new tokens into a paged cache;
  * ``kv4_read``      gives cached tokens back in BF16;
  * ``kv4_attention`` attends from new tokens (one, a few, a prompt) to the cache, and can add
    up the attention weight that every cached token has received;
  * ``kv4_evict``     keeps, per head, the tokens with the most accumulated weight next to the
    first and the last ones, and moves them to new pages.

``run`` computes them in plain torch operations in 32 bits, or (``own``) through the
framework's public functions. ``exact`` computes the same in 64 bits from the definition.

Cache. ``cache`` is uint8 [pages, kv_heads, page_size / 16, record]; a record holds 16 tokens of
one head: K codes, K parameters, V codes, V parameters. With D the head size, group g of D / g
groups and B = D / 32:
  * K codes, 8 D bytes: token t's 32-bit word c B + s (c < 4, s < B) at byte (t B 4 + word) 4 holds
    dims 32 s + 8 c + 0..7, the even ones in the low half's nibbles, the odd ones in the high
    half's;
  * K parameters, 64 D / g bytes: word 16 j + t is group j's BF16 scale (low half) and minimum;
  * V codes, 8 D bytes: word ((t / 2) 8 + r) B + b holds dims 32 b + 4 r + 0..3 of token t, of the
    even token in the low half and of the odd one in the high half;
  * V parameters as K's.
A value is code * scale + minimum; a group's scale is bf16((max - min) / 15), its minimum
bf16(min), a code clamp(round((x - minimum) / scale), 0, 15), 0 where the scale is 0.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def _join(values):
    return ",".join(str(int(v)) for v in values)


def _ints(text):
    return [int(v) for v in str(text).split(",")]


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spaced over their logarithm, in a mixed order."""
    vals = [int(round(lo * (hi / lo) ** (i / max(n - 1, 1)))) for i in range(n)]
    step = next(s for s in (7, 5, 3, 11, 13) if math.gcd(s, n) == 1)
    return [vals[(i * step) % n] for i in range(n)]


def _shape(heads, kv_heads, head_dim, group, page):
    return {"heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "group": group,
            "page": page}


LLAMA = dict(heads=32, kv_heads=8, head_dim=128)   # Llama-3-8B attention
QWEN = dict(heads=12, kv_heads=2, head_dim=128)    # Qwen2.5-1.5B attention


def listed():
    return [
        # one decode step of a small model: latency is all there is
        {"name": "append_1x1_qwen", "op": "append", "lens": "301", "new": "1",
         **_shape(**QWEN, group=64, page=16)},
        # prompts of mixed lengths entering the cache together, two of them behind a prefix
        {"name": "append_prompts_llama", "op": "append",
         "lens": "4096,1,37,2049,803,1500", "new": "4096,1,37,1023,803,611",
         **_shape(**LLAMA, group=128, page=64)},
        # the smallest attention call: one sequence, one token, a short cache
        {"name": "decode_b1_qwen", "op": "attention", "lens": "513", "new": "1",
         "weights": False, "lse": True, **_shape(**QWEN, group=64, page=16)},
        # a serving batch of ragged lengths, an empty slot and a first token among them
        {"name": "decode_b32_ragged_llama", "op": "attention",
         "lens": _join([0, 1] + _spread(30, 17, 4096)), "new": _join([1] * 32),
         "weights": False, "lse": False, **_shape(**LLAMA, group=64, page=64)},
        # one long context, where the work has to be split along the cache
        {"name": "decode_b1_128k_llama", "op": "attention", "lens": "131072", "new": "1",
         "weights": False, "lse": True, **_shape(**LLAMA, group=128, page=256)},
        # a full serving batch that tracks the attention weight of every cached token
        {"name": "decode_b64_8k_weights_llama", "op": "attention",
         "lens": _join([8192 - 61 * (i % 8) for i in range(64)]), "new": _join([1] * 64),
         "weights": True, "lse": False, **_shape(**LLAMA, group=64, page=64)},
        # a few drafted tokens a sequence to be checked in one call, small heads, fine groups
        {"name": "draft5_b16_d64", "op": "attention", "lens": _join(_spread(16, 300, 3001)),
         "new": _join([5] * 16), "weights": False, "lse": True,
         **_shape(heads=16, kv_heads=4, head_dim=64, group=32, page=32)},
        # a fresh prompt
        {"name": "prompt_4k_llama", "op": "attention", "lens": "4096", "new": "4096",
         "weights": False, "lse": False, **_shape(**LLAMA, group=64, page=64)},
        # ragged prompts that also leave the weights an eviction reads
        {"name": "prompts_weights_qwen", "op": "attention", "lens": "2999,1021,517,65",
         "new": "2999,1021,517,65", "weights": True, "lse": True,
         **_shape(**QWEN, group=128, page=64)},
        # a chunk of a long prompt against what is cached before it
        {"name": "chunk_512_of_16k_llama", "op": "attention", "lens": "16384", "new": "512",
         "weights": False, "lse": False, **_shape(**LLAMA, group=64, page=64)},
        # eviction after the prompts
        {"name": "evict_b8_8k_to_2k_llama", "op": "evict", "lens": _join([8192] * 7 + [8000]),
         "budget": 2048, "first": 4, "recent": 512, **_shape(**LLAMA, group=64, page=64)},
        # eviction of short ragged caches, one of them within the budget
        {"name": "evict_small_d64", "op": "evict", "lens": "700,257,90", "budget": 256,
         "first": 1, "recent": 33, **_shape(heads=4, kv_heads=2, head_dim=64, group=64,
                                            page=16)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    shape = rng.choice([_shape(**LLAMA, group=0, page=0), _shape(**QWEN, group=0, page=0),
                        _shape(16, 4, 64, 0, 0), _shape(8, 8, 128, 0, 0), _shape(14, 2, 64, 0, 0)])
    shape["group"] = rng.choice([g for g in (32, 64, 128) if g <= shape["head_dim"]])
    shape["page"] = rng.choice([16, 32, 64, 128, 256])
    kind = rng.choice(["append", "decode", "decode", "decode", "draft", "prompt", "prompt",
                       "chunk", "evict"])
    if kind == "append":
        batch = _log(rng, 1, 16)
        new = [_log(rng, 1, 8192 // batch) for _ in range(batch)]
        lens = [n + rng.choice([0, _log(rng, 1, 2000)]) for n in new]
        return {"op": "append", "lens": _join(lens), "new": _join(new), **shape}
    if kind == "evict":
        batch = _log(rng, 1, 8)
        top = _log(rng, 200, 8192)
        lens = [max(1, int(top * rng.uniform(0.3, 1.0))) for _ in range(batch)]
        budget = max(16, int(top * rng.uniform(0.1, 0.6)))
        first = rng.choice([0, 1, 4])
        recent = int((budget - first) * rng.uniform(0.0, 0.8))
        return {"op": "evict", "lens": _join(lens), "budget": budget, "first": first,
                "recent": recent, **shape}
    weights = rng.random() < 0.4
    if kind == "decode":
        batch = _log(rng, 1, 64)
        top = _log(rng, 40, min(131072, 64 * 8000 // batch))
        lens = [max(1, int(top * rng.uniform(0.2, 1.0))) for _ in range(batch)]
        new = [1] * batch
    elif kind == "draft":
        batch = _log(rng, 1, 16)
        top = _log(rng, 100, 8000)
        new = [rng.randint(1, 12) for _ in range(batch)]
        lens = [n + max(1, int(top * rng.uniform(0.2, 1.0))) for n in new]
    elif kind == "prompt":
        batch = _log(rng, 1, 4)
        new = [_log(rng, 33, 4000 // batch) for _ in range(batch)]
        lens = list(new)
    else:
        batch = _log(rng, 1, 2)
        new = [_log(rng, 16, 500 // batch) for _ in range(batch)]
        lens = [n + _log(rng, 500, 15000 // batch) for n in new]
    return {"op": "attention", "lens": _join(lens), "new": _join(new), "weights": weights,
            "lse": True, **shape}


# --------------------------------------------------------------------------------------
# the record layout, for the plain form (units of 16 bits)
# --------------------------------------------------------------------------------------
def _record_bytes(D, group):
    return 16 * (D + 8 * (D // group))


def _token_rows(table, page, n):
    """Record number (page * page_size / 16 + record in the page, counted without heads) and row
    in the record of positions n (int64) of one sequence, as (page, record, row)."""
    pages = table[n // page].long()
    return pages, (n % page) // 16, n % 16


def _write(cache, where, k_codes, k_scale, k_min, v_codes, v_scale, v_min, group):
    """Store quantized tokens: where = (page, record, row) of each of T tokens; codes int32
    [T, H, D], scales and minimums bf16 [T, H, D / group]."""
    T, H, D = k_codes.shape
    G, B = D // group, D // 32
    half = cache.view(torch.int16)
    flat = half.view(-1)
    R16 = half.shape[-1]
    page, rec, row = where
    heads = torch.arange(H, device=cache.device)
    base = (((page[:, None] * H + heads) * half.shape[2]) + rec[:, None]) * R16   # [T, H]
    t = row[:, None, None]

    def nibbles(c4):  # [..., 4] -> the int16 with nibble i = c4[i]
        u = c4[..., 0] | (c4[..., 1] << 4) | (c4[..., 2] << 8) | (c4[..., 3] << 12)
        return torch.where(u >= 32768, u - 65536, u).to(torch.int16)

    # K: dims (s, c, i, half) -> int16s (c, s, half) of nibbles i
    kc = k_codes.view(T, H, B, 4, 4, 2).permute(0, 1, 3, 2, 5, 4)
    kw = nibbles(kc).reshape(T, H, D // 4)
    flat[(base[..., None] + t * (D // 4) + torch.arange(D // 4, device=cache.device))] = kw
    # V: dims (b, r, i) -> int16s (r, b) of nibbles i
    vc = v_codes.view(T, H, B, 8, 4).permute(0, 1, 3, 2, 4)
    vw = nibbles(vc).reshape(T, H, D // 4)
    vbase = 4 * D + 32 * G
    off = vbase + (t // 2) * (D // 2) + 2 * torch.arange(D // 4, device=cache.device) + t % 2
    flat[base[..., None] + off] = vw
    g = torch.arange(G, device=cache.device)
    for start, sc, mn in ((4 * D, k_scale, k_min), (vbase + 4 * D, v_scale, v_min)):
        p = base[..., None] + start + 2 * (16 * g + t)
        flat[p] = sc.contiguous().view(torch.int16)
        flat[p + 1] = mn.contiguous().view(torch.int16)


def _quantize(x, group):
    """bf16 [T, H, D] -> codes int32 [T, H, D], scales and minimums bf16 [T, H, D / group]."""
    T, H, D = x.shape
    f = x.float().reshape(T, H, D // group, group)
    mx, mn = f.amax(-1), f.amin(-1)
    # divided by a tensor: a division by a Python number may become a product
    scale = ((mx - mn) / torch.full_like(mx, 15.0)).to(torch.bfloat16)
    low = mn.to(torch.bfloat16)
    s, m = scale.float()[..., None], low.float()[..., None]
    q = torch.round((f - m) / torch.where(s == 0, torch.ones_like(s), s)).clamp(0, 15)
    q = torch.where(s == 0, torch.zeros_like(q), q)
    return q.to(torch.int32).view(T, H, D), scale, low


def _unpack(rec, D, group):
    """Records uint8 [H, R, record] of one sequence -> K, V fp32 [H, 16 R, D]."""
    H, R = rec.shape[:2]
    G, B = D // group, D // 32
    half = rec.view(torch.int16)
    shift = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device=rec.device)

    def params(start):
        p = half[..., start:start + 32 * G].contiguous().view(torch.bfloat16)
        p = p.view(H, R, G, 16, 2).float()
        p = p.permute(0, 1, 3, 2, 4).reshape(H, 16 * R, G, 2)
        return p[..., 0:1], p[..., 1:2]

    def nibbles(h16):
        return ((h16.to(torch.int32)[..., None] >> shift) & 15).float()

    kc = nibbles(half[..., :4 * D].reshape(H, R * 16, 4, B, 2))          # c, s, half, i
    kc = kc.permute(0, 1, 3, 2, 5, 4).reshape(H, 16 * R, G, group)
    vbase = 4 * D + 32 * G
    vc = nibbles(half[..., vbase:vbase + 4 * D].reshape(H, R * 8, 8, B, 2))  # r, b, token, i
    vc = vc.permute(0, 1, 4, 3, 2, 5).reshape(H, 16 * R, G, group)
    ks, km = params(4 * D)
    vs, vm = params(vbase + 4 * D)
    return ((kc * ks + km).view(H, 16 * R, D), (vc * vs + vm).view(H, 16 * R, D))


def _sequence(cache, table_row, n, D, group):
    """K, V fp32 [H, n, D] of the first n tokens of a sequence."""
    page = cache.shape[2] * 16
    pages = table_row[:(n + page - 1) // page].long()
    rec = cache[pages].permute(1, 0, 2, 3).reshape(cache.shape[1], -1, cache.shape[3])
    rec = rec[:, :(n + 15) // 16]
    k, v = _unpack(rec, D, group)
    return k[:, :n], v[:, :n]


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _keys_values(gen, T, H, D, channel):
    """Keys with a few channels that are much wider than the others, as projections with a
    rotation have them; values without."""
    k = torch.randn(T, H, D, generator=gen, device=DEV) * channel
    v = torch.randn(T, H, D, generator=gen, device=DEV) * 0.7
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _offsets(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    H, D, group, page = case["kv_heads"], case["head_dim"], case["group"], case["page"]
    lens = _ints(case["lens"])
    batch = len(lens)
    width = max(1, max((n + page - 1) // page for n in lens))
    need = [(n + page - 1) // page for n in lens]
    out_pages = 0
    if case["op"] == "evict":
        out_pages = (case["budget"] + page - 1) // page
    total = sum(need) + batch * out_pages + 3
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(batch, width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = torch.zeros(total, H, page // 16, _record_bytes(D, group), dtype=torch.uint8,
                        device=DEV)
    channel = 0.5 + torch.rand(H, D, generator=gen, device=DEV)
    wide = torch.rand(H, D, generator=gen, device=DEV) < 0.04
    channel = torch.where(wide, channel * 4, channel)
    state = {"case": dict(case), "cache": cache, "table": table, "lens_list": lens,
             "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "max_len": max(lens)}
    new = _ints(case["new"]) if "new" in case else [0] * batch
    state["new_list"] = new
    for b, n in enumerate(lens):
        filled = n - new[b] if case["op"] == "append" else n
        for lo in range(0, filled, 16384):
            pos = torch.arange(lo, min(filled, lo + 16384), device=DEV)
            k, v = _keys_values(gen, pos.numel(), H, D, channel)
            _write(cache, _token_rows(table[b], page, pos), *_quantize(k, group),
                   *_quantize(v, group), group)
    if case["op"] == "append":
        state["starts"] = _offsets(new)
        state["k"], state["v"] = _keys_values(gen, sum(new), H, D, channel)
        state["weights"] = torch.ones(batch, H, width * page, device=DEV)
    elif case["op"] == "attention":
        state["starts"] = _offsets(new)
        state["max_new"] = max(new)
        q = torch.randn(sum(new), case["heads"], D, generator=gen, device=DEV)
        state["q"] = q.to(torch.bfloat16)
        state["scale"] = D ** -0.5
        if case["weights"]:
            state["weights"] = torch.rand(batch, H, width * page, generator=gen, device=DEV)
            state["weights_out"] = torch.zeros_like(state["weights"])
        if own:
            import gemv_w4a16_group_gb300 as w4
            state["workspace"] = torch.zeros(w4.kv4_attention_workspace_bytes(
                batch, sum(new), max(new), max(lens), case["heads"], H, D, group,
                case["weights"]), dtype=torch.uint8, device=DEV)
    else:
        # accumulated weight is steep: a few tokens hold most of it, some were never attended
        w = torch.rand(batch, H, width * page, generator=gen, device=DEV).pow(6) * 30
        state["weights"] = torch.where(w < 1e-6, torch.zeros_like(w), w)
        budget = case["budget"]
        state["out_table"] = order[at:at + batch * out_pages].view(batch, out_pages).clone()
        kept = [min(n, budget) for n in lens]
        state["kept_list"] = kept
        state["starts"] = _offsets(kept)
        state["weights_out"] = torch.zeros(batch, H, out_pages * page, device=DEV)
    return state


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _run_append(state)
    if op == "attention":
        return _run_attention(state)
    return _run_evict(state)


def _run_append(st):
    """The new tokens go into the cache; what it now holds of them is read back, as a program
    does whose own prompt attention has to see the values that later steps will see."""
    c = st["case"]
    group = c["group"]
    if own:
        import gemv_w4a16_group_gb300 as w4
        w4.kv4_append(st["cache"], st["table"], st["lens"], st["starts"], st["k"], st["v"],
                      group=group, weights=st["weights"])
        k, v = w4.kv4_read(st["cache"], st["table"], st["lens"], st["starts"],
                           st["k"].shape[0], c["head_dim"], group=group)
        return {"k": k, "v": v, "weights": st["weights"]}
    parts, at = [], 0
    for b, (n, m) in enumerate(zip(st["lens_list"], st["new_list"])):
        pos = torch.arange(n - m, n, device=DEV)
        parts.append(_token_rows(st["table"][b], c["page"], pos))
        st["weights"][b, :, n - m:n] = 0
        at += m
    where = tuple(torch.cat([p[i] for p in parts]) for i in range(3))
    _write(st["cache"], where, *_quantize(st["k"], group), *_quantize(st["v"], group), group)
    ks, vs = [], []
    for b, (n, m) in enumerate(zip(st["lens_list"], st["new_list"])):
        k, v = _sequence(st["cache"], st["table"][b], n, c["head_dim"], group)
        ks.append(k[:, n - m:].transpose(0, 1))
        vs.append(v[:, n - m:].transpose(0, 1))
    return {"k": torch.cat(ks).to(torch.bfloat16), "v": torch.cat(vs).to(torch.bfloat16),
            "weights": st["weights"]}


def _run_attention(st):
    c = st["case"]
    if own:
        import gemv_w4a16_group_gb300 as w4
        lse = None
        if c["lse"]:
            lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
        out = w4.kv4_attention(
            st["q"], st["cache"], st["table"], st["lens"], st["starts"], st["max_len"],
            st["max_new"], group=c["group"], scale=st["scale"], lse=lse,
            weights=st.get("weights"), weights_out=st.get("weights_out"),
            workspace=st["workspace"])
        res = {"out": out}
        if c["lse"]:
            res["lse"] = lse
        if c["weights"]:
            res["weights"] = st["weights_out"]
        return res
    H, D, G = c["kv_heads"], c["head_dim"], c["heads"] // c["kv_heads"]
    outs, lses, at = [], [], 0
    for b, (n, m) in enumerate(zip(st["lens_list"], st["new_list"])):
        q = st["q"][at:at + m].float()
        at += m
        if n == 0:
            outs.append(torch.zeros(m, c["heads"], D, dtype=torch.bfloat16, device=DEV))
            lses.append(torch.full((m, c["heads"]), -math.inf, device=DEV))
            continue
        k, v = _sequence(st["cache"], st["table"][b], n, D, c["group"])
        got = torch.zeros(H, n, device=DEV)
        cols = torch.arange(n, device=DEV)
        for lo in range(0, m, 512):
            hi = min(m, lo + 512)
            qq = q[lo:hi].view(hi - lo, H, G, D).permute(1, 2, 0, 3).reshape(H, -1, D)
            s = (qq @ k.transpose(1, 2)).view(H, G, hi - lo, n) * st["scale"]
            pos = torch.arange(n - m + lo, n - m + hi, device=DEV)
            hide = cols > pos[:, None]
            s = s.masked_fill(hide, -math.inf)
            top = s.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            e = torch.exp(s - top)
            z = e.sum(-1, keepdim=True)
            p = e / torch.where(z == 0, torch.ones_like(z), z)
            if c["weights"]:
                got += p.sum((1, 2))
            o = p.view(H, -1, n) @ v
            outs.append(o.view(H, G, hi - lo, D).permute(2, 0, 1, 3)
                        .reshape(hi - lo, c["heads"], D).to(torch.bfloat16))
            lses.append((top + torch.log(z)).view(H * G, hi - lo).transpose(0, 1))
        if c["weights"]:
            st["weights_out"][b, :, :n] = st["weights"][b, :, :n] + got
    res = {"out": torch.cat(outs)}
    if c["lse"]:
        res["lse"] = torch.cat(lses).contiguous()
    if c["weights"]:
        res["weights"] = st["weights_out"]
    return res


def _run_evict(st):
    """The tokens that stay are moved to the new pages; the cache there is given back as the
    values it holds."""
    c = st["case"]
    budget, first, recent, group = c["budget"], c["first"], c["recent"], c["group"]
    if own:
        import gemv_w4a16_group_gb300 as w4
        kept, new_lens, weights = w4.kv4_evict(
            st["cache"], st["table"], st["lens"], st["weights"], st["out_table"], budget,
            st["max_len"], c["head_dim"], first=first, recent=recent, group=group,
            weights_out=st["weights_out"])
        k, v = w4.kv4_read(st["cache"], st["out_table"], new_lens, st["starts"],
                           sum(st["kept_list"]), c["head_dim"], group=group)
        return {"kept": kept, "lens": new_lens, "weights": weights, "k": k, "v": v}
    H, page = c["kv_heads"], c["page"]
    batch = len(st["lens_list"])
    kept = torch.full((batch, H, budget), -1, dtype=torch.int32, device=DEV)
    half = st["cache"].view(torch.int16)
    flat = half.view(-1)
    rows, R16 = half.shape[2], half.shape[3]
    D, G = c["head_dim"], c["head_dim"] // group
    ks, vs = [], []
    for b, n in enumerate(st["lens_list"]):
        w = st["weights"][b, :, :n]
        m = min(n, budget)
        if n > budget:
            rank = w.clone()
            rank[:, :first] = math.inf
            rank[:, n - recent:] = math.inf
            idx = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :budget]
            idx = torch.sort(idx, dim=1).values
        else:
            idx = torch.arange(n, device=DEV).expand(H, n)
        kept[b, :, :m] = idx
        st["weights_out"][b, :, :m] = torch.gather(w, 1, idx)
        to = torch.arange(m, device=DEV)
        heads = torch.arange(H, device=DEV)[:, None]

        def address(table_row, pos):   # [H, m] -> record base and row, 16-bit units
            pages = table_row[pos // page].long()
            return ((pages * H + heads) * rows + (pos % page) // 16) * R16, pos % 16

        src, st_row = address(st["table"][b], idx)
        dst, dt_row = address(st["out_table"][b], to.expand(H, m))
        vbase = 4 * D + 32 * G
        lane = torch.arange(D // 4, device=DEV)
        pair = torch.arange(2 * G, device=DEV)
        for part in range(4):
            def at(base, row):
                row = row[..., None]
                if part == 0:
                    off = row * (D // 4) + lane
                elif part == 1:
                    off = vbase + (row // 2) * (D // 2) + 2 * lane + row % 2
                else:
                    off = (4 * D if part == 2 else vbase + 4 * D)
                    off = off + 2 * (16 * (pair // 2) + row) + pair % 2
                return base[..., None] + off
            flat[at(dst, dt_row)] = flat[at(src, st_row)]
        k, v = _sequence(st["cache"], st["out_table"][b], m, D, group)
        ks.append(k.transpose(0, 1))
        vs.append(v.transpose(0, 1))
    new_lens = torch.clamp(st["lens"], max=budget)
    return {"kept": kept, "lens": new_lens, "weights": st["weights_out"],
            "k": torch.cat(ks).to(torch.bfloat16), "v": torch.cat(vs).to(torch.bfloat16)}


# --------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------
def work(case):
    H, D = case["kv_heads"], case["head_dim"]
    token = H * _record_bytes(D, case["group"]) // 16     # a cached token, all heads
    lens = _ints(case["lens"])
    if case["op"] == "append":
        T = sum(_ints(case["new"]))
        values = 2 * T * H * D
        return {"bytes": values * 2 + T * token + T * H * 4 + values * 2, "flops": values * 7}
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        moved = kept * token * 2 + kept * H * (4 + 4)
        return {"bytes": sum(lens) * H * 4 + moved + 2 * kept * H * D * 2,
                "flops": 2 * 2 * kept * H * D}
    new = _ints(case["new"])
    pairs = 0
    for n, m in zip(lens, new):
        lo = max(0, n - m)          # the first row sees lo + 1 tokens, the last n
        pairs += (lo + 1 + n) * (n - lo) // 2
    T = sum(new)
    nbytes = T * case["heads"] * D * 2 * 2 + sum(lens) * token
    if case["lse"]:
        nbytes += T * case["heads"] * 4
    if case["weights"]:
        nbytes += sum(lens) * H * 8
    return {"bytes": nbytes, "flops": 4 * D * case["heads"] * pairs}


# --------------------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------------------
def _exact_tables(D, group):
    """For dim d of the token in row t: byte and shift of its K and V codes, byte of its
    parameters."""
    t = torch.arange(16)[:, None]
    d = torch.arange(D)[None, :]
    blocks, groups = D // 32, D // group
    kb = t * (D // 2) + 4 * (((d % 32) // 8) * blocks + d // 32) + 2 * (d % 2) + (d % 8) // 4
    k_shift = (4 * (((d % 8) // 2) % 2)).expand(16, D)
    kp = 8 * D + 4 * (16 * (d // group) + t)
    v0 = 8 * D + 64 * groups
    vb = v0 + 4 * (((t // 2) * 8 + (d % 32) // 4) * blocks + d // 32) + 2 * (t % 2) + (d % 4) // 2
    v_shift = (4 * ((d % 4) % 2)).expand(16, D)
    return kb, k_shift, kp, vb, v_shift, v0 + kp


def _exact_values(st, table_row, n, head):
    """K and V of one head of a sequence, fp64 [n, D]."""
    c = st["case"]
    cache, D = st["cache"], c["head_dim"]
    tabs = [x.to(DEV) for x in _exact_tables(D, c["group"])]
    count = (n + 15) // 16
    per_page = cache.shape[2]
    r = torch.arange(count, device=DEV)
    rec = cache[table_row.long()[r // per_page], head, r % per_page]      # [records, bytes]

    def half(at):
        bits = (rec[:, at].to(torch.int32) | (rec[:, at + 1].to(torch.int32) << 8)) << 16
        return bits.view(torch.float32).double()

    res = []
    for cb, shift, pb in (tabs[0:3], tabs[3:6]):
        code = ((rec[:, cb].to(torch.int32) >> shift) & 15).double()
        res.append((code * half(pb) + half(pb + 2)).reshape(count * 16, D)[:n])
    return res


def _exact_quantized(x, group):
    """The values that bf16 [T, H, D] becomes; the format fixes its steps in 32 bits."""
    T, H, D = x.shape
    f = x.float().reshape(T, H, D // group, group)
    low = f.min(-1, keepdim=True).values
    span = f.max(-1, keepdim=True).values - low
    scale = torch.div(span, torch.full_like(span, 15)).bfloat16().double()
    low = low.bfloat16().double()
    step = torch.where(scale == 0, torch.ones_like(scale), scale)
    code = ((f - low.float()) / step.float()).round().clamp(0, 15).double()
    code = torch.where(scale == 0, torch.zeros_like(code), code)
    return (code * scale + low).reshape(T, H, D)


def exact(case, seed):
    st = prepare(case, seed)
    H, D, heads = case["kv_heads"], case["head_dim"], case["heads"]
    lens = st["lens_list"]
    if case["op"] == "append":
        w = st["weights"].double()
        for b, (n, m) in enumerate(zip(lens, st["new_list"])):
            w[b, :, n - m:n] = 0
        return {"k": _exact_quantized(st["k"], case["group"]),
                "v": _exact_quantized(st["v"], case["group"]), "weights": w}
    if case["op"] == "evict":
        budget, first, recent = case["budget"], case["first"], case["recent"]
        total = sum(st["kept_list"])
        w_out = st["weights_out"].double()
        k_out = torch.zeros(total, H, D, dtype=torch.float64, device=DEV)
        v_out = torch.zeros_like(k_out)
        at = 0
        for b, n in enumerate(lens):
            m = min(n, budget)
            for h in range(H):
                w = st["weights"][b, h, :n].double()
                idx = torch.arange(n, device=DEV)
                if n > budget:
                    free = idx[first:n - recent]
                    best = torch.argsort(-w[free], stable=True)[:budget - first - recent]
                    idx = torch.cat([idx[:first], free[best].sort().values, idx[n - recent:]])
                w_out[b, h, :m] = w[idx]
                k, v = _exact_values(st, st["table"][b], n, h)
                k_out[at:at + m, h] = k[idx]
                v_out[at:at + m, h] = v[idx]
            at += m
        return {"kept": None, "lens": None, "weights": w_out, "k": k_out, "v": v_out}
    G = heads // H
    out = torch.zeros(sum(st["new_list"]), heads, D, dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    w_out = st["weights_out"].double() if case["weights"] else None
    at = 0
    for b, (n, m) in enumerate(zip(lens, st["new_list"])):
        for h in range(H if n else 0):
            k, v = _exact_values(st, st["table"][b], n, h)
            seen = torch.zeros(n, dtype=torch.float64, device=DEV)
            for head in range(h * G, (h + 1) * G):
                for lo in range(0, m, 2048):
                    hi = min(m, lo + 2048)
                    x = st["q"][at + lo:at + hi, head].double() @ k.T * st["scale"]
                    last = torch.arange(n - m + lo, n - m + hi, device=DEV)
                    x[torch.arange(n, device=DEV)[None, :] > last[:, None]] = -math.inf
                    z = torch.logsumexp(x, 1)
                    p = torch.exp(x - z[:, None])
                    out[at + lo:at + hi, head] = p @ v
                    lse[at + lo:at + hi, head] = z
                    seen += p.sum(0)
            if case["weights"]:
                w_out[b, h, :n] = st["weights"][b, h, :n].double() + seen
        at += m
    res = {"out": out}
    if case["lse"]:
        res["lse"] = lse
    if case["weights"]:
        res["weights"] = w_out
    return res
