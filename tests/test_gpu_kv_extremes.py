"""Attention over the cache where scores or values go to extremes: scores of -inf and far beyond those of
models, values whose sizes and weights lie far apart."""
import numpy as np
import pytest
import torch

import kv_ref as kr
from group_wise_bit_amd import qlin
from test_gpu_kv import dev, host, new_cache, new_table

pytestmark = pytest.mark.gpu


def put(cache, ref, table, k, v, counts):
    """Rows of k and v as the sequences' tokens; the reference is given what the library wrote."""
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    lengths = np.asarray(counts, np.int32)
    qlin.kv_write(cache, dev(k.astype(np.float16)), dev(v.astype(np.float16)), dev(table), dev(lengths),
                  starts=dev(starts))
    ref.data[:] = host(cache.data).reshape(ref.data.shape)
    return lengths


def widened(table, width):
    """The same pages in a table of more places (above 1024 tokens sequences are split)."""
    out = np.full((len(table), width), -1, np.int32)
    out[:, :table.shape[1]] = table
    return out


@pytest.mark.parametrize("vb", [4, 16])
@pytest.mark.parametrize("scale", [0.125, 0.7, 1.0, -1.0, 30.0])
@pytest.mark.parametrize("width", [6, 40])
def test_scores_without_end(vb, scale, width):
    """Keys of -inf (kept with 16 bits) give scores of -inf, which weigh nothing: in a wave's first
    tiles, in later ones, in single tokens, in all of a row's."""
    rng = np.random.default_rng(21)
    cache, ref = new_cache(rng, 24, 1, 64, 32, 16, vb)
    table = new_table(rng, 4, 6, 24)
    counts = [170, 170, 170, 170]
    k, v = rng.uniform(-1, 1, (680, 1, 64)), rng.standard_normal((680, 1, 64))
    pos = np.arange(680) % 170
    seq = np.arange(680) // 170
    gone = np.select([seq == 0, seq == 1, seq == 2], [pos < 128, (pos >= 64) & (pos < 150), pos % 7 < 5], True)
    k[gone, 0, 5] = -np.inf * np.sign(scale)
    lengths = put(cache, ref, table, k, v, counts)
    q = rng.uniform(0.5, 1, (4, 3, 64)).astype(np.float16)
    o, o16, lse = qlin.kv_attention(cache, dev(q), dev(widened(table, width)), dev(lengths), scale=scale,
                                    want_lse=True)
    o, o16, lse = host(o), host(o16), host(lse)
    # the definition: over the tokens whose scores are finite
    for b in range(3):
        here = ~gone[seq == b]
        sub, sub_ref = new_cache(rng, 6, 1, 64, 32, 16, vb)
        n = put(sub, sub_ref, np.arange(6, dtype=np.int32)[None], k[seq == b][here], v[seq == b][here],
                [int(here.sum())])
        want, wl, eo, el = kr.attention(sub_ref, q[b:b + 1], np.arange(6)[None], n, scale, 0)
        kr.check(o[b:b + 1], want, eo, ("O", b))
        kr.check16(o16[b:b + 1], want, eo, ("O16", b))
        kr.check(lse[b:b + 1], wl, el, ("lse", b))
    assert not o[3].any() and not o16[3].any() and np.isneginf(lse[3]).all()


@pytest.mark.parametrize("width", [6, 40])
def test_infinite_queries(width):
    """A query of inf on keys below 0 scores -inf everywhere: zeros, and only in its own rows."""
    rng = np.random.default_rng(22)
    cache, ref = new_cache(rng, 6, 1, 64, 32, 16, 8)
    table = new_table(rng, 1, 6, 6)
    k, v = -rng.uniform(0.5, 1, (150, 1, 64)), rng.standard_normal((150, 1, 64))
    lengths = put(cache, ref, table, k, v, [150])
    q = rng.uniform(-1, 1, (1, 3, 64)).astype(np.float16)
    q[0, 1, 3] = np.inf
    o, _, lse = qlin.kv_attention(cache, dev(q), dev(widened(table, width)), dev(lengths), scale=1.0,
                                  want_lse=True)
    o, lse = host(o), host(lse)
    assert not o[0, 1].any() and np.isneginf(lse[0, 1])
    rest = [0, 2]
    want, wl, eo, el = kr.attention(ref, q[:, rest], table, lengths, 1.0, 0)
    kr.check(o[:, rest], want, eo, "O")
    kr.check(lse[:, rest], wl, el, "lse")


@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (16, 16)])
@pytest.mark.parametrize("scale", [2.0 ** 20, -2.0 ** 20, 2.0 ** 12, 16.0, 1.0])
@pytest.mark.parametrize("width", [6, 40])
def test_far_scores(kb, vb, scale, width):
    """Scores of any size the arguments allow.  Keys and queries are whole numbers that the cache
    holds exactly (a group's range is 15 or 255 steps of 1), so that fp32 holds every score
    q . k < 2^24 and their differences, and a weight is wrong by the rounding of its own
    exponent only: 4 U relative to |S - max S|, which is 40 at most where it counts."""
    rng = np.random.default_rng(23)
    seqs, n = 3, 170
    cache, ref = new_cache(rng, 6 * seqs, 1, 128, 32, kb, vb)
    table = new_table(rng, seqs, 6, 6 * seqs)
    low, high = (-7, 8) if kb == 4 else (-127, 128)
    k = rng.integers(low, high + 1, (seqs * n, 1, 128)).astype(float)
    k[:, :, ::64], k[:, :, 1::64] = low, high
    # tokens that score the same as another, by 1 less, and by 2 less
    for b in range(seqs):
        for i, at in enumerate((40, 41, 90, 169)):
            k[b * n + at] = k[b * n + 11]
            k[b * n + at, 0, 2] += (i % 3) * (-1 if k[b * n + 11, 0, 2] > 0 else 1)
    v = rng.uniform(-2, 2, (seqs * n, 1, 128))
    lengths = put(cache, ref, table, k, v, [n] * seqs)
    q = np.round(rng.integers(-200, 201, (seqs, 3, 128)))
    q[:, :, 2] = 1
    for b in range(seqs):                        # one query that token 11 scores highest on
        q[b, 2] = np.sign(scale) * np.clip(k[b * n + 11, 0] * 3, -300, 300)
        q[b, 2, 2] = 1
    q = q.astype(np.float16)
    o, o16, lse = qlin.kv_attention(cache, dev(q), dev(widened(table, width)), dev(lengths), scale=scale,
                                    want_lse=True)
    o, o16, lse = host(o), host(o16), host(lse)
    for b in range(seqs):
        kk, vv = ref.sequence(table, b, 0, n)
        assert np.array_equal(kk[:, 0], k[b * n:(b + 1) * n, 0])
        for h in range(3):
            x = kk[:, 0] @ q[b, h].astype(float)
            assert (np.abs(kk[:, 0]) @ np.abs(q[b, h].astype(float))).max() < 2 ** 24
            s = scale * x
            p = np.exp(s - s.max())
            total = p.sum()
            want = (p / total) @ vv[:, 0]
            err = (p / total) @ np.abs(vv[:, 0]) * (2 * kr.U * (4 * 40 + n + 64) + 2.0 ** -20) + \
                n * 2.0 ** -38 * np.abs(vv).max()
            kr.check(o[b, h], want, err, ("O", b, h))
            kr.check16(o16[b, h], want, err, ("O16", b, h))
            wl = s.max() + np.log(total)
            kr.check(lse[b, h], wl, (n + 64) * kr.U + 8 * kr.U * (abs(wl) + 1), ("lse", b, h))


def from_dim_0(cache, ref, q, table, lengths):
    """(O, lse, their bounds) of queries that are 0 but in dim 0, with a scale of 1: a score is one
    exact product.  A weight's exponent is rounded relative to S - max S, and once more for every
    rise of the running maximum, 18 U of it in all.  A wave has tiles / 4 + 1 tiles at most; each adds
    64 roundings of its products' sums, 8 of the weights', 8 of factors; exp, the waves' sums, parts
    of other work-groups and the division add 100 + 2 tiles.  P s (P alone with 16 bits) is held to 21 bits and a step of 2^-39 of the row's
    largest, P * 2^-24 at least, |q - z| <= qmax.  The codes of a group reach from 0 or 1 to qmax or
    qmax - 1, so that its largest value is 7 s (127 s) at least and s qmax below 2.5 times that, s's
    rounding to fp16 included."""
    eo, el = np.zeros(q.shape), np.zeros(q.shape[:2])
    o, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in range(len(q)):
        k, v = (x[:, 0] for x in ref.sequence(table, b, 0, int(lengths[b])))
        n, sizes = len(k), np.abs(v).max(-1)
        for h in range(q.shape[1]):
            s = k[:, 0] * float(q[b, h, 0])
            p = np.exp(s - s.max())
            tiles = -(-n // 32)
            e = kr.U * (18 * (s.max() - s) + 80 * (tiles / 4 + 1) + 100 + 2 * tiles)
            lse[b, h] = s.max() + np.log(p.sum())
            p /= p.sum()
            o[b, h] = p @ v
            el[b, h] = p @ e + 8 * kr.U * (abs(lse[b, h]) + 1)
            step = 2.0 ** -38 * p.max() * sizes.max() if ref.bits[1] == 16 else \
                2.0 ** -39 * max((p * 2.5 * sizes).max(), p.max() * 2.0 ** -24 * 255)
            eo[b, h] = (p * (e + p @ e + 2.0 ** -20)) @ np.abs(v) + n * step
    return o, lse, eo, el


@pytest.mark.parametrize("vb", [4, 8])
@pytest.mark.parametrize("far", [12.0, 25.0, 40.0, 70.0])
@pytest.mark.parametrize("width", [6, 40])
def test_large_values_of_little_weight(vb, far, width):
    """Tokens of large values whose scores lie far below, first, last, between others and alone in
    a wave's tiles, do not cost the others their bits."""
    rng = np.random.default_rng(24)
    places = [[0], [31], [169], [3, 40, 100, 130], list(range(32, 64)), list(range(128, 170))]
    seqs, n = len(places), 170
    cache, ref = new_cache(rng, 6 * seqs, 1, 128, 32, 16, vb)
    table = new_table(rng, seqs, 6, 6 * seqs)
    k = rng.standard_normal((seqs * n, 1, 128))
    v = 1.2e-4 * rng.uniform(-1, 1, (seqs * n, 1, 128))
    k[:, :, 0] *= 0.1
    for b, at in enumerate(places):
        for i in at:
            k[b * n + i, 0, 0] = -far
            v[b * n + i] = rng.choice([-6e4, 5e4, 6e4], (1, 128))
    lengths = put(cache, ref, table, k, v, [n] * seqs)
    q = np.zeros((seqs, 3, 128), np.float16)
    q[:, :, 0] = 1, 0.5, 0.25
    o, _, lse = qlin.kv_attention(cache, dev(q), dev(widened(table, width)), dev(lengths), scale=1.0,
                                  want_lse=True)
    want, wl, eo, el = from_dim_0(cache, ref, q, table, lengths)
    kr.check(host(o), want, eo, "O")
    kr.check(host(lse), wl, el, "lse")


@pytest.mark.parametrize("vb", [4, 8])
@pytest.mark.parametrize("far", [5.0, 30.0, 60.0])
def test_weight_on_tokens_without_values(vb, far):
    """Where the highest scores are those of tokens whose values are zeros, or are small, the
    output comes from the others."""
    rng = np.random.default_rng(25)
    n = 170
    for small in (0.0, 1e-4):
        for at in ([0], [169], [5, 77], list(range(96, 128))):
            cache, ref = new_cache(rng, 6, 1, 64, 32, 16, vb)
            table = new_table(rng, 1, 6, 6)
            k, v = rng.standard_normal((n, 1, 64)), rng.uniform(-2, 2, (n, 1, 64))
            k[:, :, 0] *= 0.1
            k[at, 0, 0] = far
            v[at] *= small
            lengths = put(cache, ref, table, k, v, [n])
            q = np.zeros((1, 4, 64), np.float16)
            q[:, :, 0] = 1, 0.5, 0.25, 0
            for width in (6, 40):
                o, _, lse = qlin.kv_attention(cache, dev(q), dev(widened(table, width)), dev(lengths),
                                              scale=1.0, want_lse=True)
                want, wl, eo, el = from_dim_0(cache, ref, q, table, lengths)
                kr.check(host(o), want, eo, ("O", small, at[0], width))
                kr.check(host(lse), wl, el, ("lse", small, at[0], width))


@pytest.mark.parametrize("vb", [4, 8, 16])
@pytest.mark.parametrize("step", [0.3, -0.3, 2.0, -2.0])
def test_scores_that_climb(vb, step):
    """Scores that rise or fall from token to token, and values that do the reverse."""
    rng = np.random.default_rng(26)
    n = 1300
    cache, ref = new_cache(rng, 41, 1, 64, 32, 16, vb)
    table = new_table(rng, 1, 41, 41)
    k, v = rng.standard_normal((n, 1, 64)), rng.uniform(-1, 1, (n, 1, 64))
    k[:, 0, 0] = (step * np.arange(n)) % 700.0
    v *= np.exp(-np.minimum((abs(step) * np.arange(n)) % 20.0, 9.0))[:, None, None]
    lengths = put(cache, ref, table, k, v, [n])
    q = np.zeros((1, 2, 64), np.float16)
    q[:, :, 0] = 1, -0.5
    o, _, lse = qlin.kv_attention(cache, dev(q), dev(table), dev(lengths), scale=1.0, want_lse=True)
    want, wl, eo, el = from_dim_0(cache, ref, q, table, lengths)
    kr.check(host(o), want, eo, "O")
    kr.check(host(lse), wl, el, "lse")


def test_weights_are_rounded_to_either_side():
    """Values that are 1 in a dim of their token's own add up to 1 over the dims, but for the rounding
    of P to its two halves and that of the sums: 4 U at most, to either side, so that the mean of 512
    rows is off by 16 U / sqrt(512) < U at four standard errors."""
    rng = np.random.default_rng(27)
    seqs, heads, n = 16, 32, 61
    cache, ref = new_cache(rng, 2 * seqs, 1, 64, 32, 16, 16)
    table = new_table(rng, seqs, 2, 2 * seqs)
    k = rng.standard_normal((seqs * n, 1, 64))
    v = np.tile(np.eye(64)[:n, None], (seqs, 1, 1))
    lengths = put(cache, ref, table, k, v, [n] * seqs)
    q = rng.standard_normal((seqs, heads, 64)).astype(np.float16)
    o = host(qlin.kv_attention(cache, dev(q), dev(table), dev(lengths), scale=0.1)[0]).astype(np.float64)
    assert abs((o.sum(-1) - 1).mean()) <= kr.U


@pytest.mark.parametrize("vb", [4, 8, 16])
@pytest.mark.parametrize("width", [6, 40])
def test_values_and_scores_that_are_not_finite(vb, width):
    """An infinite value shows in its own dims (its group's where it is quantized) and a score of
    +inf in its own row; what is beside them keeps its bits, large values of the same token too."""
    rng = np.random.default_rng(28)
    n = 170
    cache, ref = new_cache(rng, 6, 1, 128, 32, 16, vb)
    table = new_table(rng, 1, 6, 6)
    k, v = rng.uniform(0.5, 1, (n, 1, 128)), rng.uniform(-1, 1, (n, 1, 128))
    v[20, 0, :64] *= 3e4
    v[20, 0, 70] = np.inf
    lengths = put(cache, ref, table, k, v, [n])
    q = rng.uniform(-0.2, 0.2, (1, 4, 128)).astype(np.float16)
    q[0, 2, 3] = np.inf
    o, _, lse = qlin.kv_attention(cache, dev(q), dev(widened(table, width)), dev(lengths), scale=1.0,
                                  want_lse=True)
    o, lse = host(o), host(lse)
    rows, bad = [0, 1, 3], np.arange(128) >= 64 if vb < 16 else np.arange(128) == 70
    assert not np.isfinite(o[0, 2]).any() and not np.isfinite(o[0, rows][:, bad]).any()
    # (the reference without the group that is not finite: its values as zeros)
    clean = v.copy()
    clean[20, 0, 64:] = 0
    sub, sub_ref = new_cache(rng, 6, 1, 128, 32, 16, vb)
    put(sub, sub_ref, table, k, clean, [n])
    want, wl, eo, el = kr.attention(sub_ref, q[:, rows], table, lengths, 1.0, 0)
    kr.check(o[:, rows][:, :, :64], want[:, :, :64], eo[:, :, :64], "O")
    kr.check(lse[:, rows], wl, el, "lse")
