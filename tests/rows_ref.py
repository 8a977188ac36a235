"""64-bit references and error bounds of the row-wise products (routing,
experts, adapters), from their definitions.

Bounds count roundings: u32 = 2^-24 and u16 = 2^-11 are the half steps of fp32
and fp16 relative to the value, 2^-25 the half step of fp16's subnormals.  A
sum of fp32 products over k terms, in any order, is within (k + 8) u32 of
sum |term| (one rounding per addition, the group's scale and the work-group's
reduction included)."""
import math

import numpy as np

import oracle

U32, U16, SUB16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -25


def route_ref(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_top=1,
              renormalize=True, scale=1.0):
    """(ids, weights in binary64) row by row."""
    m, experts = logits.shape
    top_groups = groups if top_groups is None else top_groups
    ids = np.full((m, top_k), -1, np.int32)
    wts = np.zeros((m, top_k))
    per = experts // groups
    big = float(np.finfo(np.float32).max)
    for i in range(m):
        l = {e: min(float(v), big) for e, v in enumerate(logits[i])
             if not math.isnan(v) and v != -math.inf}
        if score == "softmax":
            top = max(l.values(), default=0.0)
            tot = math.fsum(math.exp(v - top) for v in l.values())
            p = {e: math.exp(v - top) / tot for e, v in l.items()}
        else:
            p = {e: (1 / (1 + math.exp(-v)) if v > -700 else 0.0) for e, v in l.items()}
        live = [e for e in l if bias is None or float(bias[e]) > -math.inf]
        b = {e: p[e] + (float(bias[e]) if bias is not None else 0.0) for e in live}
        key = b if bias is not None else {e: l[e] for e in live}
        keep = range(groups)
        if groups > 1:
            val = {}
            for g in range(groups):
                src = key if group_top == 1 else b
                best = sorted((src[e] for e in live if e // per == g), reverse=True)[:group_top]
                if best:
                    val[g] = math.fsum(best) if all(map(math.isfinite, best)) else sum(best)
            keep = sorted(val, key=lambda g: (-val[g], g))[:top_groups]
        chosen = sorted((e for e in live if e // per in keep), key=lambda e: (-key[e], e))[:top_k]
        tot = math.fsum(p[e] for e in chosen) if renormalize else 1.0
        for j, e in enumerate(chosen):
            ids[i, j] = e
            wts[i, j] = scale * (p[e] / tot if tot > 0 else 0.0)
    return ids, wts


def silu(g):
    return g / (1.0 + np.exp(-g))


def moe_ref(x, gate, up, down, ids, wts):
    """(Y, bound of |Y_fp32 - Y|) in binary64; gate, up, down: dequantized [E, n, k]."""
    m, top_k = ids.shape
    experts, inner, model = gate.shape
    x = x.astype(np.float64)
    y = np.zeros((m, model))
    err = np.zeros((m, model))
    mag = np.zeros((m, model))
    gk, gi = (model + 8) * U32, (inner + 8) * U32
    for j in range(top_k):
        for i in range(m):
            e = int(ids[i, j])
            if not 0 <= e < experts:
                continue
            xi, ax = x[i], np.abs(x[i])
            g, u = gate[e] @ xi, up[e] @ xi
            eg, eu = gk * (np.abs(gate[e]) @ ax), gk * (np.abs(up[e]) @ ax)
            h = silu(g) * u
            # silu' <= 1.1; silu evaluated with 1-ulp exp and reciprocal: 4e-6 relative;
            # one rounding to fp16
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 4e-6 * np.abs(h)
            eh = eh + U16 * (np.abs(h) + eh) + SUB16
            d = down[e] @ h
            ed = np.abs(down[e]) @ eh + gi * (np.abs(down[e]) @ (np.abs(h) + eh))
            w = float(wts[i, j])
            y[i] += w * d
            err[i] += abs(w) * ed
            mag[i] += abs(w) * (np.abs(d) + ed)
    # the weight's product and the slots' additions
    return y, err + (top_k + 2) * U32 * mag


def lora_ref(x, what, a, b, scale, ids):
    """(Y, bound of |Y_fp32 - Y|) in binary64."""
    m, k = x.shape
    slots, rank, _ = a.shape
    x64 = x.astype(np.float64)
    y = x64 @ what.T
    err = (k + 8) * U32 * (np.abs(x64) @ np.abs(what).T)
    mag = np.abs(y)
    for i in range(m):
        s = int(ids[i])
        if not 0 <= s < slots:
            continue
        sc = float(scale[s]) if scale is not None else 1.0
        a64, b64 = a[s].astype(np.float64), b[s].astype(np.float64)
        t = sc * (a64 @ x64[i])
        # the first product in fp32, times the scale; then 22 bits of the row's largest entry
        et = abs(sc) * (k + 16) * U32 * (np.abs(a64) @ np.abs(x64[i])) + 2 * U32 * np.abs(t)
        et = et + 2.0 ** -22 * (np.abs(t) + et) + 2.0 ** -36 * np.max(np.abs(t) + et)
        y[i] += b64 @ t
        err[i] += np.abs(b64) @ et + (2 * rank + 8) * U32 * (np.abs(b64) @ (np.abs(t) + et))
        mag[i] += np.abs(b64) @ np.abs(t)
    return y, err + 4 * U32 * (mag + err)


def half_bound(y, err):
    """Bound of the fp16 output: the fp32 one's, rounded once."""
    return err + U16 * (np.abs(y) + err) + SUB16


def check_half(got, ref, err, label):
    """The fp16 output: the fp32 one's bound, rounded once.  fp16's largest value is
    65504 = 2^16 - 32 and its step there 32, so nearest-even rounding takes |v| >= 65520 to
    infinity: an infinity of the right sign is right where |ref| + err reaches 65520, and
    needed where |ref| - err does."""
    got = got.astype(np.float64)
    inf = np.isinf(got)
    assert np.all(np.where(inf, np.abs(ref) + err >= 65520, np.abs(ref) - err < 65520)), label
    assert np.array_equal(np.sign(got[inf]), np.sign(ref[inf])), label
    check(np.where(inf, ref, got), ref, half_bound(ref, err), label)


def check(got, ref, bound, label):
    got = got.astype(np.float64)
    off = np.abs(got - ref)
    bad = ~(off <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, off - bound, -np.inf))), off.shape)
        raise AssertionError(f"{label}: {bad.sum()} of {off.size} outside; at {i} got {got[i]!r} "
                             f"want {ref[i]!r} off {off[i]:.3e} > {bound[i]:.3e}")


def packed_stack(rng, count, n, k, bits, group, std=0.02):
    """(words, scales, zeros of the stack, dequantized [count, n, k]) of random masters."""
    words, scales, zeros, what = [], [], [], []
    for _ in range(count):
        w16 = (rng.standard_normal((n, k), dtype=np.float32) * np.float32(std)).astype(np.float16)
        codes, s16, z = oracle.quantize(w16, bits, group)
        words.append(oracle.pack_codes(codes, bits).view(np.int32).reshape(-1))
        scales.append(oracle.tile_meta(s16).reshape(-1))
        zeros.append(oracle.tile_meta(z).reshape(-1))
        what.append(oracle.dequantize(codes, s16, z, group))
    return (np.concatenate(words), np.concatenate(scales), np.concatenate(zeros), np.stack(what))
