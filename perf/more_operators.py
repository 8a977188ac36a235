"""Operators of a decode step around its products: the quantized cache of keys and values (writing
new tokens into its pages, reading them back, attention of one new token per sequence over it), and
drawing the next token from the logits.

Each case is one pass of one operator.  With `own` false the pass is the operator's plain form in
elementary torch operations; with `own` true it is the call a user of the library makes.
"""
import math

import numpy as np
import torch

own = False

TILE = 32                       # tokens of a cache tile
GROUP = 64                      # values per scale and zero point


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of each running sequence enters the cache: latency
        dict(name="store decode batch", op="store", seqs=48, new=1, length=2000, spread="ragged",
             kv_heads=8, head_dim=128, k_bits=4, v_bits=4, page=64, dtype="fp16", pad=0),
        # chunks of a few prompts behind cached prefixes, ragged, with padding rows behind the last
        dict(name="store odd chunks", op="store", seqs=5, new=409, length=1500, spread="ragged",
             kv_heads=2, head_dim=64, k_bits=8, v_bits=8, page=32, dtype="fp32", pad=37),
        # whole prompts of several requests
        dict(name="store prompts", op="store", seqs=8, new=2048, length=2048, spread="equal",
             kv_heads=8, head_dim=128, k_bits=8, v_bits=4, page=64, dtype="fp16", pad=0),
        # a cached prefix of one request is read back for its next chunk's dense attention
        dict(name="read prefix", op="read", seqs=1, length=1031, spread="equal", kv_heads=8,
             head_dim=128, k_bits=4, v_bits=4, page=64, dtype="fp16"),
        # the cached prompts of a batch, ragged
        dict(name="read prompts", op="read", seqs=16, length=4096, spread="ragged", kv_heads=8,
             head_dim=128, k_bits=8, v_bits=8, page=128, dtype="fp16"),
        # one token of a small model with a short history: latency
        dict(name="attend token", op="attend", seqs=1, length=333, spread="equal", heads=14,
             kv_heads=2, head_dim=64, k_bits=8, v_bits=8, page=64, window=0, out="fp16"),
        # a serving batch, lengths from one token to thousands
        dict(name="attend decode batch", op="attend", seqs=48, length=4096, spread="ragged",
             heads=32, kv_heads=8, head_dim=128, k_bits=4, v_bits=4, page=64, window=0, out="fp16"),
        # one very long sequence
        dict(name="attend long", op="attend", seqs=1, length=131071, spread="equal", heads=32,
             kv_heads=8, head_dim=128, k_bits=4, v_bits=4, page=128, window=0, out="fp16"),
        # unquantized cache, a sliding window, one wide head of keys for all queries
        dict(name="attend window", op="attend", seqs=9, length=6000, spread="ragged", heads=20,
             kv_heads=1, head_dim=256, k_bits=16, v_bits=16, page=32, window=1000, out="fp32"),
        # a full card of long sequences
        dict(name="attend long batch", op="attend", seqs=64, length=8192, spread="equal", heads=32,
             kv_heads=8, head_dim=128, k_bits=8, v_bits=8, page=64, window=0, out="fp16"),
        # the next token of one request
        dict(name="sample token", op="sample", m=1, vocab=151936, temperature=True, top_k=True,
             top_p=True, min_p=False, rounded=False, masked=0.0),
        # a serving batch, each request with its own settings, a grammar's mask, logits with ties
        dict(name="sample decode batch", op="sample", m=64, vocab=151936, temperature=True,
             top_k=True, top_p=True, min_p=True, rounded=True, masked=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("store", "read", "attend", "attend", "attend", "sample"))
    if op == "sample":
        m = _log(rng, 1, 64)
        return dict(op=op, m=m, vocab=_log(rng, 1000, 151936), temperature=rng.random() < 0.8,
                    top_k=rng.random() < 0.6, top_p=rng.random() < 0.6, min_p=rng.random() < 0.4,
                    rounded=rng.random() < 0.5, masked=rng.choice((0.0, 0.3)))
    head_dim = rng.choice((64, 128, 128, 256))
    c = dict(op=op, kv_heads=rng.choice((1, 2, 4, 8)), head_dim=head_dim,
             k_bits=rng.choice((4, 8, 16)), v_bits=rng.choice((4, 8, 16)),
             page=rng.choice((32, 64, 128, 256)), spread=rng.choice(("equal", "ragged")))
    if op == "attend":
        while True:
            c.update(seqs=_log(rng, 1, 64), length=_log(rng, 1, 131072),
                     window=rng.choice((0, 0, 0, _log(rng, 1, 4096))),
                     out=rng.choice(("fp16", "fp32")))
            c["heads"] = c["kv_heads"] * rng.randint(1, 20)
            whole = dict(c, window=0, spread="equal")
            if work(whole)["bytes"] <= 5e8 and c["seqs"] * c["length"] * c["kv_heads"] * head_dim <= 2 ** 28:
                return c
    c["dtype"] = rng.choice(("fp16", "fp32"))
    while True:
        c.update(seqs=_log(rng, 1, 48), length=_log(rng, 1, 16384))
        if op == "store":
            c.update(new=min(c["length"], _log(rng, 1, 4096)), pad=rng.choice((0, 0, 21)))
        rows = c["seqs"] * (c["new"] if op == "store" else c["length"])
        if rows * c["kv_heads"] * head_dim <= 2 ** 24 and \
                c["seqs"] * c["length"] * c["kv_heads"] * head_dim <= 2 ** 27:
            return c


def _lengths(c):
    """Lengths of the case's sequences: all equal, or spread from 1 to the longest."""
    n, longest = c["seqs"], c["length"]
    if c["spread"] == "equal":
        return [longest] * n
    return [1 + int((longest - 1) * ((0.31 + i * 0.6180339887498949) % 1.0) ** 2) if i else longest
            for i in range(n)]


def _counts(c):
    """Tokens of each sequence that a store writes or a read reads."""
    lengths = _lengths(c)
    if c["op"] == "read":
        return lengths
    if c["spread"] == "equal" or c["new"] == 1:
        return [min(c["new"], x) for x in lengths]
    return [min(x, 1 + (c["new"] - 1) * (3 + 5 * (i % 3)) // 13) if i else min(c["new"], x)
            for i, x in enumerate(lengths)]


def _token_bytes(c):
    """Cache bytes of one token and one head of keys and values."""
    d = c["head_dim"]
    return sum(d * b / 8 + (3 * d // GROUP if b < 16 else 0) for b in (c["k_bits"], c["v_bits"]))


def work(case):
    c = case
    if c["op"] == "sample":
        return {"bytes": 4 * c["m"] * c["vocab"] + 28 * c["m"], "flops": 4 * c["m"] * c["vocab"]}
    h, d = c["kv_heads"], c["head_dim"]
    if c["op"] == "attend":
        seen = sum(min(x, c["window"]) if c["window"] else x for x in _lengths(c))
        out = 4 if c["out"] == "fp32" else 2
        return {"bytes": seen * h * _token_bytes(c) + c["seqs"] * c["heads"] * ((2 + out) * d + 4),
                "flops": 4 * seen * c["heads"] * d}
    rows = sum(_counts(c))
    values = rows * h * d
    wide = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "read":
        return {"bytes": rows * h * _token_bytes(c) + 2 * wide * values, "flops": 4 * values}
    # written from fp16, and given back as it stands in the cache
    return {"bytes": (2 + wide) * 2 * values + rows * h * _token_bytes(c), "flops": 16 * values}


# --------------------------------------------------- a cache tile, value by value
_MAPS = {}


def _tile_bytes(d, k_bits, v_bits):
    return 4 * d * (k_bits + v_bits) + sum(96 * (d // GROUP) for b in (k_bits, v_bits) if b < 16)


def _maps(d, k_bits, v_bits, device):
    """For keys and values: the half-word of each (token, dim) of a tile and the shift of its code
    there, the half-word of each (token, group)'s scale and the byte of its zero point."""
    key = (d, k_bits, v_bits, device)
    if key not in _MAPS:
        g = d // GROUP
        t, x = torch.meshgrid(torch.arange(TILE), torch.arange(d), indexing="ij")
        tt, gg = torch.meshgrid(torch.arange(TILE), torch.arange(g), indexing="ij")
        # keys: lane (quarter of a group, token of the half tile); its run over (half, group, 16)
        b = k_bits
        lane = (x % 64 // 16) * 16 + t % 16
        at = (t // 16 * g + x // 64) * 16 + x % 16          # code of the lane's run
        word, code = at * b // 32, at % (32 // b)
        kw = ((word // 4 * 64 + lane) * 4 + word % 4) * 2 + code % 2
        ks = code // 2 * b
        # values: lane (4 tokens, 4 dims of a group); words of two tokens
        b, n = v_bits, 16 // v_bits
        lane = (t % 16 // 4) * 16 + x % 64 // 4
        unit = x // 64 * (4 // n) + x % 4 // n
        pair = t // 16 * 2 + t % 4 // 2
        vw = ((unit * 64 + lane) * 4 + pair) * 2 + t % 2 + 2 * d * k_bits
        vs = x % 4 % n * b
        at = 2 * d * (k_bits + v_bits)                      # half-words
        place = gg * 32 + (tt % 16 // 4) * 8 + tt // 16 * 4 + tt % 4
        scales, zeros = [], []
        for bits in (k_bits, v_bits):
            scales.append(place + at)
            at += 32 * g * (bits < 16)
        at *= 2
        zeros.append((tt % 16 * 2 + tt // 16) * g + gg + at)
        at += 32 * g * (k_bits < 16)
        zeros.append(((tt % 16 // 4) * g + gg) * 8 + tt // 16 * 4 + tt % 4 + at)
        _MAPS[key] = [[m.to(device) for m in part]
                      for part in ((kw, ks, scales[0], zeros[0]), (vw, vs, scales[1], zeros[1]))]
    return _MAPS[key]


def _unpack(tiles, c):
    """fp32 keys and values [..., 32, d] of cache tiles uint8 [..., bytes]."""
    d = c["head_dim"]
    half = tiles.view(torch.int16)
    out = []
    for (w, s, sc, ze), bits in zip(_maps(d, c["k_bits"], c["v_bits"], tiles.device),
                                    (c["k_bits"], c["v_bits"])):
        raw = half[..., w.reshape(-1)]
        if bits == 16:
            out.append(raw.view(torch.float16).float().unflatten(-1, (TILE, d)))
            continue
        code = (raw >> s.reshape(-1).to(torch.int16)) & ((1 << bits) - 1)
        code = code.unflatten(-1, (TILE, d // GROUP, GROUP))
        scale = half[..., sc.reshape(-1)].view(torch.float16).unflatten(-1, (TILE, d // GROUP, 1))
        zero = tiles[..., ze.reshape(-1)].unflatten(-1, (TILE, d // GROUP, 1))
        out.append(((code.float() - zero.float()) * scale.float()).flatten(-2))
    return out


def _quantize(x, bits):
    """fp16 [..., d] -> codes int32, scale fp16, zero uint8: round to nearest over the range of a
    group's values and 0; a group that is not finite gets the scale NaN."""
    w = x.float().unflatten(-1, (-1, GROUP))
    qmax = (1 << bits) - 1
    bad = ~torch.isfinite(w).all(-1, keepdim=True)
    w = w.masked_fill(bad, 0)
    lo, hi = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
    s = ((hi - lo) / qmax).half()
    f = torch.where(s == 0, torch.ones_like(lo), s.float())
    z = torch.where(s == 0, torch.zeros_like(lo), torch.round(-lo / f).clamp_(0, qmax))
    q = torch.where(s == 0, torch.zeros_like(w), (torch.round(w / f) + z).clamp_(0, qmax))
    s = s.masked_fill(bad, float("nan"))
    return q.flatten(-2).to(torch.int32), s.squeeze(-1), z.squeeze(-1).to(torch.uint8)


def _pack(keys, values, c):
    """Cache tiles uint8 [..., bytes] of fp16 keys and values [..., 32, d]."""
    d = c["head_dim"]
    bytes_ = _tile_bytes(d, c["k_bits"], c["v_bits"])
    lead = keys.shape[:-2]
    tiles = torch.zeros(*lead, bytes_, dtype=torch.uint8, device=keys.device)
    half = tiles.view(torch.int16)
    for x, (w, s, sc, ze), bits in zip((keys, values),
                                       _maps(d, c["k_bits"], c["v_bits"], keys.device),
                                       (c["k_bits"], c["v_bits"])):
        if bits == 16:
            half[..., w.reshape(-1)] = x.flatten(-2).view(torch.int16)
            continue
        q, scale, zero = _quantize(x, bits)
        q = (q << s).flatten(-2)
        order = torch.argsort(w.reshape(-1), stable=True)   # the codes of one half-word together
        n = 16 // bits
        words = q[..., order].unflatten(-1, (-1, n)).sum(-1).to(torch.int16)
        half[..., w.reshape(-1)[order][::n]] = words
        half[..., sc.reshape(-1)] = scale.flatten(-2).view(torch.int16)
        tiles[..., ze.reshape(-1)] = zero.flatten(-2)
    return tiles


# -------------------------------------------------------------------- inputs
def _cache(c, gen, dev, lengths):
    """Pages in random order, filled with tokens; behind a sequence's end lies what was left there."""
    page, h, d = c["page"], c["kv_heads"], c["head_dim"]
    per = [-(-x // page) for x in lengths]
    width = max(per) + 2                                    # room for more tokens
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    tiles = page // TILE
    data = torch.empty(pages, h, tiles * _tile_bytes(d, c["k_bits"], c["v_bits"]),
                       dtype=torch.uint8, device=dev)
    tilted = 1.0 + 2.0 * (torch.rand(h, 1, d, generator=gen, device=dev) < 0.05)
    shift = 0.5 * torch.randn(h, 1, d, generator=gen, device=dev)
    step = max(1, (1 << 24) // (h * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        k = (torch.randn(n, h, page, d, generator=gen, device=dev) * tilted + shift).half()
        v = torch.randn(n, h, page, d, generator=gen, device=dev).half()
        data[i:i + n] = _pack(k.unflatten(2, (tiles, TILE)), v.unflatten(2, (tiles, TILE)),
                              c).flatten(2)
    # the rest of a last page: values that are no numbers
    tail = torch.full((1, h, TILE, d), float("nan"), dtype=torch.float16, device=dev)
    junk = _pack(tail, tail, c)[0]
    for i, x in enumerate(lengths):
        used = -(-(x % page) // TILE) if x % page else tiles
        if used < tiles:
            row = data[order[sum(per[:i + 1]) - 1].long()]
            row.view(h, tiles, -1)[:, used:] = junk[:, None]
    return data, table


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "sample":
        m, v = c["m"], c["vocab"]
        logits = 2.0 * torch.randn(m, v, generator=gen, device=dev)
        few = torch.rand(m, v, generator=gen, device=dev) < 1e-3
        logits += few * 5.0 * torch.rand(m, v, generator=gen, device=dev)
        if c["rounded"]:
            logits = logits.half().float()
        if c["masked"]:
            rows = torch.rand(m, 1, generator=gen, device=dev)
            off = torch.rand(m, v, generator=gen, device=dev) < c["masked"]
            logits = logits.masked_fill(off & (rows < 0.4), float("-inf"))
            logits = logits.masked_fill(off & (rows > 0.8), torch.finfo(torch.float32).min)
        s["logits"] = logits

        def setting(on, values, dtype):
            at = torch.randint(0, len(values), (m,), generator=gen, device=dev)
            return torch.tensor(values, dtype=dtype, device=dev)[at] if on else None
        s["temperature"] = setting(c["temperature"], (0.6, 0.7, 0.8, 1.0, 1.3) + (0.0,) * (m > 1),
                                   torch.float32)
        s["top_k"] = setting(c["top_k"], (20, 50, 200) + (0, 1) * (m > 1), torch.int32)
        s["top_p"] = setting(c["top_p"], (0.5, 0.8, 0.9, 0.95) + (1.0,) * (m > 1), torch.float32)
        s["min_p"] = setting(c["min_p"], (0.0, 0.02, 0.1), torch.float32)
        s["u"] = torch.rand(m, generator=gen, device=dev)
        return s
    h, d = c["kv_heads"], c["head_dim"]
    lengths = _lengths(c)
    s["data"], s["table"] = _cache(c, gen, dev, lengths)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["longest"] = max(lengths)
    if c["op"] == "attend":
        s["q"] = (1.3 * torch.randn(c["seqs"], c["heads"], d, generator=gen, device=dev)).half()
        return s
    counts = _counts(c)
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    s["rows"] = starts[-1]
    s["single"] = counts == [1] * len(counts)               # one token each: no row offsets needed
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    if c["op"] == "store":
        m = starts[-1] + c["pad"]
        s["k"] = (torch.randn(m, h, d, generator=gen, device=dev) *
                  (1.0 + 2.0 * (torch.rand(h, d, generator=gen, device=dev) < 0.05)) +
                  0.5 * torch.randn(h, d, generator=gen, device=dev)).half()
        s["v"] = torch.randn(m, h, d, generator=gen, device=dev).half()
        if m > 4:
            s["k"][m // 3, :, :GROUP] = 0                   # a group of zeros, and one of one sign
            s["v"][m // 2] = s["v"][m // 2].abs() + 1
    return s


# --------------------------------------------------------------- plain forms
def _places(s):
    """Page and offset of each row, and whether there is one."""
    c = s["case"]
    row = torch.arange(s["rows"], device=s["data"].device)
    seq = torch.searchsorted(s["starts"][1:].long(), row, right=True)
    pos = s["lengths"].long()[seq] - (s["starts"].long()[seq + 1] - row)
    page = s["table"].long()[seq, (pos // c["page"]).clamp(0, s["table"].shape[1] - 1)]
    there = (pos >= 0) & (page >= 0) & (page < s["data"].shape[0])
    return page.clamp(min=0), pos % c["page"], there


def _plain_read(s, place=None):
    c = s["case"]
    h, d = c["kv_heads"], c["head_dim"]
    page, offset, there = place or _places(s)
    data = s["data"].unflatten(2, (c["page"] // TILE, -1))
    half, t = data.view(torch.int16), offset % TILE
    head = torch.arange(h, device=page.device)[None, :, None]
    where = (page[:, None, None], head, (offset // TILE)[:, None, None])
    out = []
    for (w, sh, sc, ze), bits in zip(_maps(d, c["k_bits"], c["v_bits"], data.device),
                                     (c["k_bits"], c["v_bits"])):
        raw = half[(*where, w[t][:, None])]
        if bits == 16:
            x = raw.view(torch.float16).float()
        else:
            code = (raw.to(torch.int32) >> sh[t][:, None]) & ((1 << bits) - 1)
            scale = half[(*where, sc[t][:, None])].view(torch.float16).float()[..., None]
            zero = data[(*where, ze[t][:, None])].float()[..., None]
            x = ((code.unflatten(-1, (-1, GROUP)).float() - zero) * scale).flatten(-2)
        x = x.masked_fill(~there[:, None, None], 0)
        if c["dtype"] == "fp16" and bits < 16:
            x = x.clamp(-65504, 65504)
        out.append(x.half() if c["dtype"] == "fp16" else x)
    return tuple(out)


def _plain_store(s):
    c = s["case"]
    h, d = c["kv_heads"], c["head_dim"]
    place = _places(s)
    page, offset, there = place
    data = s["data"].unflatten(2, (c["page"] // TILE, -1))
    half, n = data.view(torch.int16), s["rows"]
    page, offset = page[there], offset[there]
    t = offset % TILE
    head = torch.arange(h, device=page.device)[None, :, None]
    where = (page[:, None, None], head, (offset // TILE)[:, None, None])
    for x, (w, sh, sc, ze), bits in zip((s["k"], s["v"]),
                                        _maps(d, c["k_bits"], c["v_bits"], data.device),
                                        (c["k_bits"], c["v_bits"])):
        x = x[:n][there]
        if bits == 16:
            half[(*where, w[t][:, None])] = x.view(torch.int16)
            continue
        q, scale, zero = _quantize(x, bits)
        order = torch.argsort(w, dim=-1, stable=True)       # [32, d]
        per = 16 // bits
        q = (q << sh[t][:, None]).gather(-1, order[t][:, None].expand(-1, h, -1))
        words = q.unflatten(-1, (-1, per)).sum(-1).to(torch.int16)
        half[(*where, w.gather(-1, order)[:, ::per][t][:, None])] = words
        half[(*where, sc[t][:, None])] = scale.view(torch.int16)
        data[(*where, ze[t][:, None])] = zero
    return _plain_read(s, place)


def _plain_attend(s):
    c = s["case"]
    b, h, d, page = c["seqs"], c["kv_heads"], c["head_dim"], c["page"]
    per = -(-s["longest"] // page)
    table = s["table"][:, :per].long()
    tiles = s["data"].unflatten(2, (page // TILE, -1))[table.clamp(min=0)]
    tiles = tiles.transpose(1, 2).reshape(b, h, per * page // TILE, -1)     # [b, h, tile, bytes]
    k, v = (x.flatten(2, 3) for x in _unpack(tiles, c))
    pos = torch.arange(per * page, device=k.device)
    n = s["lengths"].long()[:, None]
    seen = (pos < n) & (table >= 0).repeat_interleave(page, 1)
    if c["window"]:
        seen &= pos >= n - c["window"]
    gone = ~seen[:, None, :]
    k, v = (x.masked_fill(gone[..., None], 0) for x in (k, v))
    q = s["q"].float().view(b, h, -1, d)
    score = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    score = score.masked_fill(gone[:, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == float("-inf"), 0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total.clamp(min=1e-38)
    lse = (top + torch.log(total)).view(b, -1)
    o = o.view(b, c["heads"], d)
    return (o if c["out"] == "fp32" else o.half()), lse


def _plain_sample(s):
    c = s["case"]
    # 64 bits: the draw goes by sums over the whole vocabulary next to a border
    x = s["logits"].double()
    m, n = x.shape
    here = ~(torch.isnan(x) | (x == float("-inf")))
    x = x.clamp(max=torch.finfo(torch.float32).max).masked_fill(~here, float("-inf"))
    order = x.sort(dim=-1, descending=True, stable=True)
    top = order.values[:, :1].clamp(min=-1e300)
    t = s["temperature"].double()[:, None] if s["temperature"] is not None else torch.ones_like(top)
    greedy = t <= 0
    mass = torch.exp((order.values - top) / t.masked_fill(greedy, 1))
    place = torch.arange(n, device=x.device)
    keep = order.values > float("-inf")
    keep &= ~greedy | (place < 1)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (k <= 0) | (place < k)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        sums = torch.cumsum(mass.masked_fill(~keep, 0), -1)
        before = sums - mass.masked_fill(~keep, 0)
        keep &= (p >= 1) | (place < 1) | (before < p * sums[:, -1:])
    if s["min_p"] is not None:
        keep &= (place < 1) | (mass >= s["min_p"].double()[:, None])
    kept = torch.zeros_like(x).scatter_(1, order.indices, mass.masked_fill(~keep, 0))
    sums = torch.cumsum(kept, -1)
    total = sums[:, -1:]
    past = (sums > s["u"].double()[:, None] * total) & (kept > 0)
    last = torch.where(kept > 0, place, torch.full_like(place, -1)).amax(-1)
    first = torch.where(past, place, torch.full_like(place, n)).amin(-1)
    ids = torch.where(first < n, first, last)
    probs = kept.gather(1, ids.clamp(min=0)[:, None])[:, 0] / total[:, 0].clamp(min=1e-300)
    return ids.to(torch.int32), probs.masked_fill(ids < 0, 0).float()


# ------------------------------------------------------------ the library's calls
def _own_cache(s):
    from group_wise_bit_amd import qlin
    c = s["case"]
    if "cache" not in s:
        s["cache"] = qlin.KVCache(s["data"], c["kv_heads"], c["head_dim"], c["page"], c["k_bits"],
                                  c["v_bits"])
    return qlin, s["cache"]


def _own_read(s):
    qlin, cache = _own_cache(s)
    dtype = torch.float16 if s["case"]["dtype"] == "fp16" else torch.float32
    return qlin.kv_read(cache, s["table"], s["lengths"],
                        starts=None if s["single"] else s["starts"], rows=s["rows"], dtype=dtype)


def _own_store(s):
    qlin, cache = _own_cache(s)
    qlin.kv_write(cache, s["k"], s["v"], s["table"], s["lengths"],
                  starts=None if s["single"] else s["starts"])
    return _own_read(s)


def _own_attend(s):
    qlin, cache = _own_cache(s)
    f32 = s["case"]["out"] == "fp32"
    o, o16, lse = qlin.kv_attention(cache, s["q"], s["table"], s["lengths"],
                                    window=s["case"]["window"], want_o=f32, want_o16=not f32,
                                    want_lse=True)
    return (o if f32 else o16), lse


def _own_sample(s):
    from group_wise_bit_amd import qlin
    if "sampling" not in s:
        s["sampling"] = qlin.Sampling(temperature=s["temperature"], top_k=s["top_k"],
                                      top_p=s["top_p"], min_p=s["min_p"])
    return qlin.sample(s["sampling"], s["logits"], s["u"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"store": _own_store, "read": _own_read, "attend": _own_attend,
                "sample": _own_sample}[op](state)
    return {"store": _plain_store, "read": _plain_read, "attend": _plain_attend,
            "sample": _plain_sample}[op](state)


# ------------------------------------------------------------ 64 bits, from the definitions
def _values64(tile, c):
    """Keys and values [..., 32, d] in 64 bits of cache tiles, by the layout's rules."""
    d, g = c["head_dim"], c["head_dim"] // 64
    lead, at, codes, out = tile.shape[:-1], 0, [], []
    for bits in (c["k_bits"], c["v_bits"]):
        size = 4 * d * bits
        codes.append(tile[..., at:at + size].reshape(*lead, -1, 64, 16))     # [unit, lane, byte]
        at += size
    meta = []
    for width in (2, 1):
        for i, bits in enumerate((c["k_bits"], c["v_bits"])):
            part = tile[..., at:at + 32 * g * width] if bits < 16 else None
            at += 32 * g * width if bits < 16 else 0
            meta.append(part)
    for i, bits in enumerate((c["k_bits"], c["v_bits"])):
        n = 16 // bits
        w = codes[i].contiguous().view(torch.int16).to(torch.int64) & 0xFFFF  # [unit, lane, 8]
        q = torch.stack([(w >> (bits * j)) & ((1 << bits) - 1) for j in range(n)], -1)
        q = q.unflatten(-2, (4, 2))                          # [unit, lane, word, half, code]
        if i == 0:
            # codes in the lane's run go (unit, word, code, half); lane = (quarter, token)
            q = q.transpose(-1, -2).unflatten(-4, (4, 16))   # [unit, quarter, token, word, code, half]
            q = q.movedim(-6, -4).flatten(-4).unflatten(-1, (2, g, 16))
            q = q.movedim((-5, -4, -3, -2, -1), (-2, -4, -5, -3, -1))
        else:
            # unit = (group, part of 4 dims), lane = (4 tokens, 4 dims), word = (half tile, pair)
            q = q.unflatten(-5, (g, 4 // n)).unflatten(-4, (4, 16)).unflatten(-3, (2, 2))
            # [group, part, four, c, half tile, pair, half, code]
            q = q.movedim((-8, -7, -6, -5, -4, -3, -2, -1), (-4, -2, -7, -3, -8, -6, -5, -1))
        q = q.reshape(*lead, 32, d)
        if bits == 16:
            x = q.to(torch.int16)
            out.append(x.view(torch.float16).double())
            continue
        s = meta[i].contiguous().view(torch.float16).double().reshape(*lead, g, 4, 2, 4)
        s = s.movedim((-4, -3, -2, -1), (-1, -3, -4, -2)).reshape(*lead, 32, g, 1)
        z = meta[2 + i].double()
        if i == 0:
            z = z.reshape(*lead, 16, 2, g).transpose(-3, -2)
        else:
            z = z.reshape(*lead, 4, g, 2, 4).movedim((-4, -3, -2, -1), (-3, -1, -4, -2))
        z = z.reshape(*lead, 32, g, 1)
        out.append(((q.double().unflatten(-1, (g, 64)) - z) * s).reshape(*lead, 32, d))
    return out


def _stored64(x, bits):
    """What a row of fp16 values is in the cache, in 64 bits, rounded where the definition says."""
    w = x.double().unflatten(-1, (-1, 64))
    if bits == 16:
        return x.double()
    lo, hi = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
    top = 2 ** bits - 1
    s = ((hi - lo).float().double() / top).float().half().double()
    none = s == 0
    f = s.masked_fill(none, 1)
    z = torch.round((-lo / f).float().double()).clamp(0, top)
    q = (torch.round((w / f).float().double()) + z).clamp(0, top)
    return ((q - z) * s).masked_fill(none, 0).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "sample":
        return _exact_sample(s)
    h, d, page = c["kv_heads"], c["head_dim"], c["page"]
    lengths, table = s["lengths"].tolist(), s["table"].tolist()

    def sequence(i, first):
        """Keys and values [kv_heads, tokens, d] of sequence i from token `first` on."""
        at = first // page
        ids = [p for p in table[i][at:-(-lengths[i] // page)]]
        k, v = _values64(s["data"][ids].unflatten(2, (page // TILE, -1)), c)
        return [x.transpose(0, 1).reshape(h, -1, d)[:, first - at * page:lengths[i] - at * page]
                for x in (k, v)]
    if c["op"] == "store":
        n = s["rows"]
        return tuple(_stored64(x[:n], b) for x, b in ((s["k"], c["k_bits"]), (s["v"], c["v_bits"])))
    if c["op"] == "read":
        both = [sequence(i, 0) for i in range(c["seqs"])]
        return tuple(torch.cat([x[j].transpose(0, 1) for x in both]) for j in range(2))
    out, lses = [], []
    for i in range(c["seqs"]):
        k, v = sequence(i, max(0, lengths[i] - c["window"]) if c["window"] else 0)
        q = s["q"][i].double().view(h, -1, d)
        score = torch.bmm(q, k.transpose(1, 2).contiguous()) * d ** -0.5
        lse = torch.logsumexp(score, -1)
        out.append(torch.bmm(torch.exp(score - lse[..., None]), v.contiguous()).view(-1, d))
        lses.append(lse.view(-1))
    return torch.stack(out), torch.stack(lses)


def _exact_sample(s):
    ids, probs = [], []

    def setting(name, i, off):
        return off if s[name] is None else s[name][i].item()
    for i, row in enumerate(s["logits"].double().cpu().numpy()):
        here = np.flatnonzero(row > -np.inf)
        ranked = here[np.argsort(-row[here], kind="stable")]
        t = setting("temperature", i, 1.0)
        if ranked.size == 0 or t <= 0:
            ids.append(int(ranked[0]) if ranked.size else -1)
            probs.append(1.0 if ranked.size else 0.0)
            continue
        k, p = setting("top_k", i, 0), setting("top_p", i, 1.0)
        if k > 0:
            ranked = ranked[:k]
        mass = np.exp((row[ranked] - row[ranked[0]]) / t)
        if p < 1:
            sums = np.cumsum(mass)
            ranked = ranked[:1 + int(np.searchsorted(sums, p * sums[-1], side="left"))]
        mass = mass[:ranked.size]
        ranked = ranked[:max(1, int((mass >= setting("min_p", i, 0.0)).sum()))]
        ranked = np.sort(ranked)
        mass = np.exp((row[ranked] - row[ranked].max()) / t)
        ranked, mass = ranked[mass > 0], mass[mass > 0]
        sums = np.cumsum(mass)
        at = min(int(np.searchsorted(sums, s["u"][i].item() * sums[-1], side="right")),
                 ranked.size - 1)
        ids.append(int(ranked[at]))
        probs.append(float(mass[at] / sums[-1]))
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)
