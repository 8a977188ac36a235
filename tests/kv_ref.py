"""64-bit reference of the cache of keys and values (include/qlin_kv.h): the quantizer, the
layout of a page code by code, attention, and the bounds of its error.

Bounds count roundings: u = 2^-24 is fp32's half step relative to the value, 2^-11 and 2^-25
those of fp16 and of its subnormals."""
import numpy as np

U = 2.0 ** -24
TILE = 32


def tile_bytes(d, kb, vb):
    return 4 * d * (kb + vb) + 96 * (d // 64) * ((kb < 16) + (vb < 16))


def code_places(d, bits, values):
    """Per (token, dim) of a tile: the 32-bit word of the code and its lowest bit."""
    g = d // 64
    word, bit = np.zeros((TILE, d), np.int64), np.zeros((TILE, d), np.int64)
    for t in range(TILE):
        for x in range(d):
            h, c, y = t // 16, x // 64, x % 64
            if not values:
                lane, per = 16 * (y // 16) + t % 16, 32 // bits
                i = (h * g + c) * 16 + y % 16
                w = i // per
                word[t, x] = (w // 4 * 64 + lane) * 4 + w % 4
                bit[t, x] = 16 * (i % 2) + bits * (i % per // 2)
            else:
                lane, n = 16 * (t % 16 // 4) + y // 4, 16 // bits
                word[t, x] = ((c * (4 // n) + y % 4 // n) * 64 + lane) * 4 + 2 * h + t % 4 // 2
                bit[t, x] = 16 * (t % 2) + bits * (y % 4 % n)
    return word, bit


_PLACES = {}


def places(d, kb, vb):
    """For keys and values: byte and shift of each code's lowest bit, bytes of each
    (token, group)'s scale and zero point."""
    if (d, kb, vb) not in _PLACES:
        g, at, codes, scales, zeros = d // 64, 0, [], [], []
        for bits, values in ((kb, False), (vb, True)):
            w, b = code_places(d, bits, values)
            codes.append((at + 4 * w + b // 8, b % 8))
            at += 4 * d * bits
        t, c = np.meshgrid(np.arange(TILE), np.arange(g), indexing="ij")
        for bits in (kb, vb):
            scales.append(at + 2 * (c * 32 + t % 16 // 4 * 8 + t // 16 * 4 + t % 4))
            at += 64 * g * (bits < 16)
        zeros.append(at + (t % 16 * 2 + t // 16) * g + c)
        at += 32 * g * (kb < 16)
        zeros.append(at + ((t % 16 // 4 * g + c) * 2 + t // 16) * 4 + t % 4)
        at += 32 * g * (vb < 16)
        assert at == tile_bytes(d, kb, vb)
        _PLACES[d, kb, vb] = list(zip(codes, scales, zeros))
    return _PLACES[d, kb, vb]


def quantize(w, bits):
    """fp16 [..., d] -> codes, scale (fp16), zero [..., d / 64] by the header's formulas; every
    fl32 is one rounding of the exact value (a quotient of two fp32 numbers rounded through
    64 bits is rounded correctly)."""
    x = w.astype(np.float64).reshape(*w.shape[:-1], -1, 64)
    qmax = 2 ** bits - 1
    bad = ~np.isfinite(x).all(-1, keepdims=True)
    x = np.where(bad, 0, x)
    lo, hi = np.minimum(x.min(-1, keepdims=True), 0), np.maximum(x.max(-1, keepdims=True), 0)

    def fl(v):
        return v.astype(np.float32).astype(np.float64)
    s = fl(fl(hi - lo) / qmax).astype(np.float16)
    f = np.where(s == 0, 1, s.astype(np.float64))
    z = np.where(s == 0, 0, np.clip(np.rint(fl(-lo / f)), 0, qmax))
    q = np.where(s == 0, 0, np.clip(np.rint(fl(x / f)) + z, 0, qmax))
    s = np.where(bad, np.float16(np.nan), s)
    return (q.reshape(w.shape).astype(np.int64), s[..., 0].astype(np.float16),
            z[..., 0].astype(np.uint8))


class Cache:
    """Pages as bytes [pages, kv_heads, tiles, bytes]."""

    def __init__(self, data, d, kb, vb):
        self.d, self.bits = d, (kb, vb)
        self.data = data.reshape(*data.shape[:2], -1, tile_bytes(d, kb, vb))
        self.tiles = self.data.shape[2]

    def put(self, page, offset, head, which, w):
        """A token's keys (0) or values (1), fp16 [d], at its place."""
        tile, t, bits = self.data[page, head, offset // TILE], offset % TILE, self.bits[which]
        (byte, bit), scale, zero = places(self.d, *self.bits)[which]
        if bits == 16:
            raw = w.view(np.uint16)
            tile[byte[t]], tile[byte[t] + 1] = raw & 255, raw >> 8
            return
        q, s, z = quantize(w, bits)
        for x in range(self.d):
            keep = ~(((1 << bits) - 1) << bit[t, x]) & 255
            tile[byte[t, x]] = (tile[byte[t, x]] & keep) | (q[x] << bit[t, x])
        raw = s.view(np.uint16)
        tile[scale[t]], tile[scale[t] + 1], tile[zero[t]] = raw & 255, raw >> 8, z

    def get(self, page, offset, which):
        """All heads' keys or values of a token in 64 bits [kv_heads, d]."""
        tile, t, bits = self.data[page, :, offset // TILE], offset % TILE, self.bits[which]
        (byte, bit), scale, zero = places(self.d, *self.bits)[which]

        def half(at):
            raw = tile[:, at].astype(np.uint16) | (tile[:, at + 1].astype(np.uint16) << 8)
            return raw.view(np.float16).astype(np.float64)
        if bits == 16:
            return half(byte[t])
        q = (tile[:, byte[t]].astype(np.int64) >> bit[t]) & ((1 << bits) - 1)
        q = q.reshape(q.shape[0], -1, 64) - tile[:, zero[t]].astype(np.int64)[..., None]
        return (q * half(scale[t])[..., None]).reshape(q.shape[0], -1)

    def token(self, table, b, pos):
        """(page, offset) of a token, or None if it is not there."""
        size = self.tiles * TILE
        if pos < 0 or pos // size >= table.shape[1]:
            return None
        page = int(table[b, pos // size])
        return (page, pos % size) if 0 <= page < self.data.shape[0] else None

    def sequence(self, table, b, lo, hi):
        """Keys and values [tokens there, kv_heads, d] of positions lo .. hi - 1."""
        at = [p for p in (self.token(table, b, i) for i in range(lo, hi)) if p is not None]
        heads = self.data.shape[1]
        return [np.array([self.get(*p, w) for p in at]).reshape(len(at), heads, self.d)
                for w in (0, 1)]


def rows_of(lengths, starts, m):
    """(row, sequence, position) of a call's rows."""
    for b in range(len(lengths)):
        r0, r1 = (b, b + 1) if starts is None else (starts[b], starts[b + 1])
        for r in range(r0, min(r1, m)):
            yield r, b, int(lengths[b]) - (r1 - r)


def attention(cache, q, table, lengths, scale, window):
    """(O, lse, bound of O's error in fp32, bound of lse's): q [seqs, heads, d] fp16.

    A score is a sum of d exact products in fp32 (d + 8 roundings of sum |q k|, scales
    included) times scale, whose sign changes no size, and its exponent is rounded four times
    more, each relative to a value below |S| + |max S| + 40; exp is correct to 2 u.  P enters
    with 21 bits and a step of 2^-39 of the largest P s, sums over n tokens add n + 64
    roundings."""
    seqs, heads, d = q.shape
    o, lse = np.zeros((seqs, heads, d)), np.full((seqs, heads), -np.inf)
    eo, el = np.zeros((seqs, heads, d)), np.zeros((seqs, heads))
    for b in range(seqs):
        n = max(int(lengths[b]), 0)
        k, v = cache.sequence(table, b, max(n - window, 0) if window else 0, n)
        if not len(k):
            continue
        ratio = heads // k.shape[1]
        for h in range(heads):
            kh, vh = k[:, h // ratio], v[:, h // ratio]
            x = q[b, h].astype(np.float64)
            s, size = scale * (kh @ x), abs(scale) * (np.abs(kh) @ np.abs(x)).max()
            top = s.max()
            p = np.exp(s - top)
            total = p.sum()
            p /= total
            o[b, h], lse[b, h] = p @ vh, top + np.log(total)
            e = U * ((d + 16) * size + 4 * (2 * size + 40) + 8)
            el[b, h] = e + (len(k) + 64) * U + 4 * U * (abs(lse[b, h]) + 1)
            eo[b, h] = (p @ np.abs(vh)) * (2 * e + 2.0 ** -20 + 2 * (len(k) + 64) * U) + \
                len(k) * 2.0 ** -38 * np.abs(vh).max()
    return o, lse, eo, el


def check(got, ref, err, what):
    wrong = ~(np.abs(got.astype(np.float64) - ref) <= err)
    assert not wrong.any(), (what, int(wrong.sum()), np.abs(got - ref)[wrong].max())


def check16(got, ref, err, what):
    check(got, ref, err + 2.0 ** -11 * (np.abs(ref) + err) + 2.0 ** -25, what)
