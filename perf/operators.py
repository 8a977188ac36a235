"""Operators whose weights differ from row to row: routing to experts, the experts' gated MLP over
packed weights, and low-rank adapters of many requests beside one packed projection.

Each case is one pass of one operator.  With `own` false the pass is the operator's plain form in
elementary torch operations; with `own` true it is the call a user of the library makes.
"""
import math

import torch

own = False

BLOCK = 64                      # codes per K-block and weights per group


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the router of one generated token: latency
        dict(name="route token", op="route", m=1, experts=64, top_k=8, score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0, masked=0.0),
        # a serving batch's decode step: sigmoid scores, a bias for balance, groups of experts
        dict(name="route decode batch", op="route", m=48, experts=256, top_k=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5,
             masked=0.0),
        # a chunk of a prompt, an expert count that is no power of two, some experts masked off
        dict(name="route odd chunk", op="route", m=1021, experts=60, top_k=4, score="softmax",
             bias=False, groups=1, top_groups=1, group_top=1, renormalize=False, scale=1.0,
             masked=0.05),
        # all tokens of several long prompts
        dict(name="route prompts", op="route", m=16384, experts=256, top_k=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5,
             masked=0.0),
        # one generated token: eight experts of 64, read once each
        dict(name="experts token", op="experts", m=1, experts=64, top_k=8, hidden=2048, inner=1024,
             bits=4, group=64, down_bits=4, padded=0.0),
        # a decode batch over many small experts: most are hit by one or two rows; padding rows
        dict(name="experts decode batch", op="experts", m=27, experts=128, top_k=8, hidden=1024,
             inner=512, bits=3, group=64, down_bits=4, padded=0.1),
        # a chunk of a prompt over a few large experts at 8 bits, odd token count
        dict(name="experts odd chunk", op="experts", m=509, experts=16, top_k=2, hidden=4096,
             inner=1792, bits=8, group=64, down_bits=8, padded=0.0),
        # the tokens of several prompts at once
        dict(name="experts prompts", op="experts", m=4096, experts=32, top_k=4, hidden=2048,
             inner=1408, bits=4, group=64, down_bits=4, padded=0.0),
        # one generated token of a request with an adapter
        dict(name="adapters token", op="adapters", m=1, n=4096, k=4096, bits=4, group=64, slots=16,
             rank=16, spread="tokens", bare=0.0, out="fp32"),
        # a decode batch, every request with an adapter of its own or none; a q/k/v projection
        dict(name="adapters decode batch", op="adapters", m=40, n=6144, k=4096, bits=4, group=64,
             slots=64, rank=32, spread="tokens", bare=0.2, out="fp16"),
        # chunks of a few prompts, ragged, one scale per row of the weight, 2 bits
        dict(name="adapters odd chunk", op="adapters", m=333, n=896, k=4864, bits=2, group=0,
             slots=5, rank=8, spread="prompts", bare=0.1, out="fp32"),
        # the prompts of several requests, a large rank
        dict(name="adapters prompts", op="adapters", m=2048, n=4096, k=4096, bits=4, group=64,
             slots=8, rank=64, spread="prompts", bare=0.1, out="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "experts", "experts", "adapters", "adapters"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _log(rng, 4, 256 // groups)
        top_groups = rng.randint((groups + 1) // 2, groups)
        top_k = rng.randint(1, min(8, top_groups * (experts // groups)))
        return dict(op=op, m=_log(rng, 1, 16384), experts=experts, top_k=top_k,
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5,
                    groups=groups, top_groups=top_groups,
                    group_top=rng.choice((1, 2)) if groups > 1 else 1,
                    renormalize=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                    masked=rng.choice((0.0, 0.05)))
    if op == "experts":
        while True:
            experts = _log(rng, 4, 128)
            c = dict(op=op, m=_log(rng, 1, 4096), experts=experts,
                     top_k=rng.randint(1, min(8, experts)), hidden=64 * _log(rng, 8, 64),
                     inner=64 * _log(rng, 4, 32), bits=rng.choice((2, 3, 4, 5, 6, 7, 8)),
                     group=rng.choice((64, 64, 0)), down_bits=rng.choice((2, 3, 4, 6, 8)),
                     padded=rng.choice((0.0, 0.1)))
            top = listed()[7]
            if work(c)["flops"] <= work(top)["flops"] and \
                    c["experts"] * c["hidden"] * c["inner"] <= top["experts"] * top["hidden"] * top["inner"]:
                return c
    return dict(op=op, m=_log(rng, 1, 2048), n=_log(rng, 500, 4096), k=64 * _log(rng, 8, 64),
                bits=rng.choice((2, 3, 4, 5, 6, 7, 8)), group=rng.choice((64, 64, 0)),
                slots=_log(rng, 1, 64), rank=8 * rng.randint(1, 8),
                spread=rng.choice(("tokens", "prompts")), bare=rng.choice((0.0, 0.2)),
                out=rng.choice(("fp32", "fp16")))


def _weight_bytes(n, k, bits, group):
    return n * k * bits / 8 + 3 * n * (k // BLOCK if group == 64 else 1)


def work(case):
    c = case
    m = c["m"]
    if c["op"] == "route":
        return {"bytes": 4 * m * c["experts"] + 8 * m * c["top_k"], "flops": 4 * m * c["experts"]}
    if c["op"] == "experts":
        e, h, i = c["experts"], c["hidden"], c["inner"]
        pairs = m * c["top_k"] * (1 - c["padded"])
        used = e * (1 - (1 - c["top_k"] / e) ** (m * (1 - c["padded"])))
        per = 2 * _weight_bytes(i, h, c["bits"], c["group"]) + _weight_bytes(h, i, c["down_bits"],
                                                                             c["group"])
        return {"bytes": used * per + 4 * m * h + 8 * m * c["top_k"], "flops": 6 * pairs * h * i}
    n, k, r = c["n"], c["k"], c["rank"]
    rows = m * (1 - c["bare"])
    slots = c["slots"] * (1 - (1 - 1 / c["slots"]) ** rows) if c["spread"] == "tokens" \
        else min(c["slots"], rows)
    out = 4 if c["out"] == "fp32" else 2
    return {"bytes": _weight_bytes(n, k, c["bits"], c["group"]) + 2 * slots * r * (n + k) +
            2 * m * k + out * m * n + 4 * m, "flops": 2 * m * n * k + 2 * rows * r * (n + k)}


# ------------------------------------------------- packed codes, layout "tiled"
def _fields(bits):
    """The bit fields of a 64-code block: (first word, step between words, codes per word,
    low bit of the code, width, shift of each of the word's codes)."""
    def plain(width, low, first):
        per = 32 // width
        return [(first + w, w * per, low, width,
                 [16 * (i % 2) + width * (i // 2) for i in range(per)]) for w in range(64 // per)]

    def three(low, first):
        out = []
        for run in range(2):
            for u in range(2):
                out.append((first + 3 * run + u, 32 * run + 16 * u, low, 2,
                            [16 * (i % 2) + 2 * (i // 2) for i in range(16)]))
            shifts = []
            for c in range(32):
                u, i = c // 16, c % 16
                p, e = i // 2, i % 2
                b = (2 * p + 2 if p < 4 else 2 * (p - 4) + 3) + 16 * e
                shifts.append((b + 8) % 32 if u else b)
            out.append((first + 3 * run + 2, 32 * run, low + 2, 1, shifts))
        return out

    if bits in (2, 4, 8):
        return plain(bits, 0, 0)
    if bits == 3:
        return three(0, 0)
    return plain(4, 0, 0) + (three(4, 8) if bits == 7 else plain(bits - 4, 4, 8))


def _pack(code, bits):
    """int32 codes [..., 64] -> int32 words [..., 2 * bits]."""
    words = []
    for word, first, low, width, shifts in sorted(_fields(bits), key=lambda f: f[0]):
        part = (code[..., first:first + len(shifts)] >> low) & ((1 << width) - 1)
        words.append((part << torch.tensor(shifts, dtype=torch.int32, device=code.device))
                     .sum(-1, dtype=torch.int32))
    return torch.stack(words, -1)


_TABLES = {}


def _tables(bits, device):
    """Per code of a block: its word, shift, mask and place for each of the code's fields."""
    key = (bits, device)
    if key not in _TABLES:
        planes = {}
        for word, first, low, width, shifts in _fields(bits):
            plane = planes.setdefault(low, ([0] * 64, [0] * 64, width))
            plane[0][first:first + len(shifts)] = [word] * len(shifts)
            plane[1][first:first + len(shifts)] = shifts
        _TABLES[key] = [(torch.tensor(w, device=device),
                         torch.tensor(s, dtype=torch.int32, device=device), (1 << width) - 1, low)
                        for low, (w, s, width) in sorted(planes.items())]
    return _TABLES[key]


def _weights(gen, count, n, k, bits, group, device):
    """`count` matrices [n, k]: N(0, 0.02) fp16 masters rounded to nearest and packed, one after
    the other: dict of codes, scale, zero (tiled) and sizes."""
    tiles, kb = (n + 63) // 64, k // BLOCK
    gcount = kb if group == 64 else 1
    qmax = (1 << bits) - 1
    data = torch.empty(count, tiles, kb, 64, 2 * bits, dtype=torch.int32, device=device)
    scale = torch.empty(count, tiles, gcount, 64, dtype=torch.float16, device=device)
    zero = torch.empty(count, tiles, gcount, 64, dtype=torch.uint8, device=device)
    step = max(1, (1 << 24) // (n * k))
    for i in range(0, count, step):
        c = min(step, count - i)
        w = torch.randn(c, tiles * 64, kb, 64, generator=gen, device=device).mul_(0.02).half().float()
        dims = (-1,) if group == 64 else (-2, -1)
        lo, hi = w.amin(dims, keepdim=True), w.amax(dims, keepdim=True)
        s = ((hi - lo) / qmax).half()
        z = torch.round(-lo / s.float()).clamp_(0, qmax)
        q = (torch.round(w / s.float()) + z).clamp_(0, qmax).to(torch.int32)
        if n % 64:
            q[:, n:], s[:, n:], z[:, n:] = 0, 0, 0

        def tiled(t):
            return t.reshape(c, tiles, 64, t.shape[2], t.shape[3]).transpose(2, 3)
        data[i:i + c] = _pack(tiled(q), bits)
        scale[i:i + c] = tiled(s).squeeze(-1)
        zero[i:i + c] = tiled(z).squeeze(-1).to(torch.uint8)
    return dict(count=count, n=n, k=k, bits=bits, group=64 if group == 64 else k,
                data=data.reshape(-1), scale=scale.reshape(-1), zero=zero.reshape(-1))


def _dequantize(w, used=None):
    """fp32 [count (or the used ones), n, k] of packed weights."""
    tiles, kb, bits = (w["n"] + 63) // 64, w["k"] // BLOCK, w["bits"]
    words = w["data"].view(w["count"], tiles, kb, 64, 2 * bits)
    s = w["scale"].view(w["count"], tiles, -1, 64, 1)
    z = w["zero"].view(w["count"], tiles, -1, 64, 1)
    if used is not None:
        words, s, z = words[used], s[used], z[used]
    code = sum(((words[..., word] >> shift) & mask) << low
               for word, shift, mask, low in _tables(bits, words.device))
    v = (code - z.to(torch.int32)).float() * s.float()
    return v.transpose(2, 3).reshape(-1, tiles * 64, w["k"])[:, :w["n"]]


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    m = c["m"]
    if c["op"] == "route":
        e = c["experts"]
        s["logits"] = 1.5 * torch.randn(m, e, generator=gen, device=dev) + \
            0.5 * torch.randn(e, generator=gen, device=dev)
        if c["masked"]:
            off = torch.rand(m, e, generator=gen, device=dev) < c["masked"]
            s["logits"] = s["logits"].masked_fill(off, float("-inf"))
        s["bias"] = 0.1 * torch.randn(e, generator=gen, device=dev) if c["bias"] else None
        return s
    if c["op"] == "experts":
        e, h, i = c["experts"], c["hidden"], c["inner"]
        s["x"] = torch.randn(m, h, generator=gen, device=dev).half()
        s["gate"] = _weights(gen, e, i, h, c["bits"], c["group"], dev)
        s["up"] = _weights(gen, e, i, h, c["bits"], c["group"], dev)
        s["down"] = _weights(gen, e, h, i, c["down_bits"], c["group"], dev)
        logits = torch.randn(m, e, generator=gen, device=dev) + \
            0.3 * torch.randn(e, generator=gen, device=dev)
        top = torch.softmax(logits, -1).topk(c["top_k"])
        ids = top.indices.to(torch.int32)
        if c["padded"]:                      # padding rows of the batch go to no expert
            off = torch.rand(m, 1, generator=gen, device=dev) < c["padded"]
            ids = ids.masked_fill(off, -1)
        s["ids"] = ids.contiguous()
        s["weights"] = (top.values / top.values.sum(-1, keepdim=True)).contiguous()
        return s
    n, k, slots, r = c["n"], c["k"], c["slots"], c["rank"]
    s["x"] = torch.randn(m, k, generator=gen, device=dev).half()
    s["w"] = _weights(gen, 1, n, k, c["bits"], c["group"], dev)
    s["a"] = (torch.randn(slots, r, k, generator=gen, device=dev) / math.sqrt(k)).half()
    s["b"] = (0.2 * torch.randn(slots, n, r, generator=gen, device=dev)).half()
    s["scale"] = (2.0 * torch.rand(slots, generator=gen, device=dev) + 0.5).float()
    if c["spread"] == "tokens":              # one token of each request
        ids = torch.randint(0, slots, (m,), generator=gen, device=dev)
        off = torch.rand(m, generator=gen, device=dev) < c["bare"]
    else:                                    # the rows of a prompt stand together
        cuts = torch.sort(torch.rand(2 * slots - 1, generator=gen, device=dev)).values
        part = torch.searchsorted(cuts, (torch.arange(m, device=dev) + 0.5) / m)
        pick = torch.randint(0, slots, (2 * slots,), generator=gen, device=dev)
        ids = pick[part]
        off = (torch.rand(2 * slots, generator=gen, device=dev) < c["bare"])[part]
    s["ids"] = ids.masked_fill(off, -1).to(torch.int32).contiguous()
    return s


# --------------------------------------------------------------- plain forms
def _plain_route(s):
    c = s["case"]
    # 64 bits: scores that differ only behind the 24th bit are ordered too
    x = s["logits"].double()
    here = ~(torch.isnan(x) | (x == float("-inf")))
    x = x.clamp(max=torch.finfo(torch.float32).max).masked_fill(~here, float("-inf"))
    if c["score"] == "softmax":
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top.masked_fill(top == float("-inf"), 0))
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.where(here, 1 / (1 + torch.exp(-x)), torch.zeros_like(x))
    biased = (p + s["bias"].double() if s["bias"] is not None else p).masked_fill(~here,
                                                                                  float("-inf"))
    # without a bias the order of the scores is the order of the logits, exactly
    key = biased if s["bias"] is not None else x
    if c["groups"] > 1:
        m, g = x.shape[0], c["groups"]
        per = (key if c["group_top"] == 1 else biased).view(m, g, -1)
        best = per.sort(dim=-1, descending=True).values[..., :c["group_top"]]
        value = best[..., 0] + (best[..., 1:].masked_fill(best[..., 1:] == float("-inf"), 0)
                                .sum(-1) if c["group_top"] > 1 else 0)
        chosen = value.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros(m, g, dtype=torch.bool, device=x.device).scatter_(1, chosen, True)
        key = key.view(m, g, -1).masked_fill(~kept[..., None], float("-inf")).view(m, -1)
    order = key.sort(dim=-1, descending=True, stable=True)
    ids = order.indices[:, :c["top_k"]]
    there = order.values[:, :c["top_k"]] > float("-inf")
    w = p.gather(1, ids).masked_fill(~there, 0)
    if c["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return ids.masked_fill(~there, -1).to(torch.int32), (w * c["scale"]).float()


def _plain_experts(s):
    c = s["case"]
    m, k, e = c["m"], c["top_k"], c["experts"]
    flat = s["ids"].reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < e), flat, torch.full_like(flat, e))
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=e + 1)
    used = counts[:e].nonzero().squeeze(1)
    if used.numel() == 0:
        return s["x"].new_zeros(m, c["hidden"])
    # the rows of each used expert, padded to the longest
    room = int(counts[:e].max())
    place = torch.empty_like(flat)
    place[order] = torch.arange(m * k, device=flat.device) - (counts.cumsum(0) - counts)[flat[order]]
    there = flat < e
    slot = torch.searchsorted(used, flat.clamp(max=e - 1))[there] * room + place[there]
    token = torch.arange(m * k, device=flat.device)[there] // k
    x = torch.zeros(used.numel() * room, c["hidden"], device=flat.device)
    x[slot] = s["x"].float()[token]
    x = x.view(used.numel(), room, -1)
    g = torch.bmm(x, _dequantize(s["gate"], used).transpose(1, 2).contiguous())
    u = torch.bmm(x, _dequantize(s["up"], used).transpose(1, 2).contiguous())
    d = torch.bmm(g / (1 + torch.exp(-g)) * u,
                  _dequantize(s["down"], used).transpose(1, 2).contiguous())
    y = torch.zeros(m * k, c["hidden"], device=flat.device)
    y[there] = d.view(-1, c["hidden"])[slot]
    return (y.view(m, k, -1) * s["weights"][..., None]).sum(1).half()


def _plain_adapters(s):
    c = s["case"]
    x = s["x"].float()
    y = torch.matmul(x, _dequantize(s["w"])[0].t())
    # every row through every adapter, with the others' parts set to zero
    mine = (s["ids"][:, None] == torch.arange(c["slots"], device=x.device)).float() * s["scale"]
    t = torch.matmul(x, s["a"].float().view(-1, c["k"]).t()).view(c["m"], c["slots"], c["rank"])
    t = (t * mine[..., None]).view(c["m"], -1)
    y = y + torch.matmul(t, s["b"].float().transpose(1, 2).reshape(-1, c["n"]))
    return y if c["out"] == "fp32" else y.half()


# ------------------------------------------------------------ the library's calls
def _own_route(s):
    from group_wise_bit_amd import qlin
    c = s["case"]
    if "router" not in s:
        s["router"] = qlin.Router(c["experts"], c["top_k"], score=c["score"], bias=s["bias"],
                                  groups=c["groups"], top_groups=c["top_groups"],
                                  group_top=c["group_top"], renormalize=c["renormalize"],
                                  scale=c["scale"])
    return qlin.route(s["router"], s["logits"])


def _own_experts(s):
    from group_wise_bit_amd import qlin
    if "stacks" not in s:
        s["stacks"] = [qlin.QExperts(w["count"], w["n"], w["k"], w["bits"], w["group"], w["data"],
                                     w["scale"], w["zero"])
                       for w in (s["gate"], s["up"], s["down"])]
    return qlin.moe_mlp(*s["stacks"], s["x"], s["ids"], s["weights"], want_y=False)[1]


def _own_adapters(s):
    from group_wise_bit_amd import qlin
    if "weight" not in s:
        w = s["w"]
        s["weight"] = qlin.QWeight(w["n"], w["k"], w["bits"], w["group"], qlin.FMT_PACKED,
                                   w["data"], w["scale"], w["zero"])
        s["adapters"] = qlin.Adapters(s["a"], s["b"], s["scale"])
    f32 = s["case"]["out"] == "fp32"
    y, y16 = qlin.gemm_lora(s["weight"], s["x"], s["adapters"], s["ids"], want_y=f32,
                            want_y16=not f32)
    return y if f32 else y16


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "experts": _own_experts,
                "adapters": _own_adapters}[op](state)
    return {"route": _plain_route, "experts": _plain_experts, "adapters": _plain_adapters}[op](state)


# ------------------------------------------------------------ 64 bits, from the definitions
def _values64(w, e):
    """Matrix e of packed weights in 64 bits, code by code from the layout's rules."""
    tiles, kb, bits = -(-w["n"] // 64), w["k"] // 64, w["bits"]
    per = tiles * kb * 64 * 2 * bits
    words = (w["data"][e * per:(e + 1) * per].to(torch.int64) & 0xFFFFFFFF).view(tiles, kb, 64, -1)
    out = torch.empty(tiles, 64, kb, 64, dtype=torch.float64, device=words.device)

    def bit(word, at):
        return (words[..., word] >> at) & 1

    def small(first, width, c):              # the 1-, 2-, 4- and 8-bit arrangement
        per_word = 32 // width
        i = c % per_word
        return sum(bit(first + c // per_word, 16 * (i % 2) + width * (i // 2) + b) << b
                   for b in range(width))

    def three(first, c):
        run, rest = divmod(c, 32)
        u, i = divmod(rest, 16)
        p, odd = i // 2, i % 2
        high = (2 * p + 2 if p < 4 else 2 * (p - 4) + 3) + 16 * odd
        return small(first + 3 * run + u, 2, i) + \
            (bit(first + 3 * run + 2, (high + 8 * u) % 32) << 2)

    for c in range(64):
        if bits == 3:
            q = three(0, c)
        elif bits <= 4 or bits == 8:
            q = small(0, bits, c)
        else:
            q = small(0, 4, c) + ((three(8, c) if bits == 7 else small(8, bits - 4, c)) << 4)
        out[..., c] = q.transpose(1, 2).double()
    g = kb if w["group"] == 64 else 1
    s = w["scale"].view(-1, tiles, g, 64)[e].transpose(1, 2).double()[..., None]
    z = w["zero"].view(-1, tiles, g, 64)[e].transpose(1, 2).double()[..., None]
    return ((out - z) * s).reshape(tiles * 64, w["k"])[:w["n"]]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    m = c["m"]
    if c["op"] == "route":
        if m * c["experts"] > 1 << 22:       # row by row on the host: some seconds at most
            return None
        rows, bias = s["logits"].cpu().tolist(), s["bias"].tolist() if c["bias"] else None
        ids, weights = [], []
        for row in rows:
            there = [j for j, v in enumerate(row) if not math.isnan(v) and v != -math.inf]
            if c["score"] == "softmax":
                top = max((row[j] for j in there), default=0.0)
                total = math.fsum(math.exp(row[j] - top) for j in there)
                p = {j: math.exp(row[j] - top) / total for j in there}
            else:
                p = {j: 1 / (1 + math.exp(-row[j])) for j in there}
            biased = {j: p[j] + (bias[j] if bias else 0.0) for j in there}
            rank = biased if bias else {j: row[j] for j in there}
            size = c["experts"] // c["groups"]
            value = {}
            for g in range(c["groups"]):
                inside = sorted((biased[j] for j in there if j // size == g), reverse=True)
                if inside:
                    value[g] = sum(inside[:c["group_top"]])
            best = sorted(value, key=lambda g: (-value[g], g))[:c["top_groups"]]
            kept = sorted((j for j in there if j // size in best), key=lambda j: (-rank[j], j))
            kept = kept[:c["top_k"]]
            total = math.fsum(p[j] for j in kept) if c["renormalize"] else 1.0
            w = [c["scale"] * p[j] / total if total else 0.0 for j in kept]
            pad = c["top_k"] - len(kept)
            ids.append(kept + [-1] * pad)
            weights.append(w + [0.0] * pad)
        return [torch.tensor(ids, dtype=torch.int32), torch.tensor(weights, dtype=torch.float64)]
    x = s["x"].double()
    if c["op"] == "experts":
        y = torch.zeros(m, c["hidden"], dtype=torch.float64, device=x.device)
        for e in range(c["experts"]):
            token, slot = (s["ids"] == e).nonzero(as_tuple=True)
            if token.numel() == 0:
                continue
            g = x[token] @ _values64(s["gate"], e).T
            h = g * torch.sigmoid(g) * (x[token] @ _values64(s["up"], e).T)
            y.index_add_(0, token, s["weights"][token, slot].double()[:, None] *
                         (h @ _values64(s["down"], e).T))
        return y
    y = x @ _values64(s["w"], 0).T
    for a in range(c["slots"]):
        token = (s["ids"] == a).nonzero().squeeze(1)
        y[token] += s["scale"][a].double() * ((x[token] @ s["a"][a].double().T)
                                              @ s["b"][a].double().T)
    return y
