"""The cache of keys and values on a GPU: pages byte for byte, rows read back, attention of one
token per sequence, each against the 64-bit reference of tests/kv_ref.py."""
import numpy as np
import pytest
import torch

import kv_ref as kr
from group_wise_bit_amd import qlin

pytestmark = pytest.mark.gpu
DEV = "cuda"
BITS = [(4, 4), (8, 8), (16, 16), (4, 8), (8, 4), (16, 4), (4, 16), (8, 16), (16, 8)]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def new_cache(rng, pages, heads, d, page, kb, vb):
    """Pages of random bytes: (the library's cache, the reference over a copy)."""
    size = qlin.kv_page_bytes(d, page, kb, vb)
    assert size == page // 32 * kr.tile_bytes(d, kb, vb)
    data = rng.integers(0, 256, (pages, heads, size), dtype=np.uint8)
    return qlin.KVCache(dev(data), heads, d, page, kb, vb), kr.Cache(data.copy(), d, kb, vb)


def new_table(rng, seqs, width, pages):
    """Pages of their own for every sequence, in random order."""
    return rng.permutation(pages)[:seqs * width].reshape(seqs, width).astype(np.int32)


def tokens(rng, m, heads, d):
    k = rng.standard_normal((m, heads, d)) * rng.choice([0.01, 1.0, 30.0], (m, heads, 1))
    v = rng.standard_normal((m, heads, d))
    for x in (k, v):
        if m > 2:
            x[1, :, :64] = np.abs(x[1, :, :64]) + 2       # one sign
            x[2, :, :64] = -np.abs(x[2, :, :64]) - 1
        if m > 4:
            x[3, :, :64] = 0
            x[4, :, :64] = 5e-8 * rng.integers(-3, 4, 64)  # fp16's smallest numbers
    return k.astype(np.float16), v.astype(np.float16)


def store(ref, k, v, table, lengths, starts):
    for r, b, pos in kr.rows_of(lengths, starts, len(k)):
        at = ref.token(table, b, pos)
        if at is not None:
            for h in range(k.shape[1]):
                ref.put(*at, h, 0, k[r, h])
                ref.put(*at, h, 1, v[r, h])


def fill(rng, cache, ref, table, lengths):
    """Every sequence's tokens written in one call; the reference is given what the library wrote."""
    starts = np.concatenate([[0], np.cumsum(np.maximum(lengths, 0))]).astype(np.int32)
    k, v = tokens(rng, max(int(starts[-1]), 1), cache.kv_heads, cache.head_dim)
    k = np.clip(k, -8, 8).astype(np.float16)
    qlin.kv_write(cache, dev(k), dev(v), dev(table), dev(lengths), starts=dev(starts))
    ref.data[:] = host(cache.data).reshape(ref.data.shape)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kb,vb", BITS)
def test_write_pages(d, kb, vb):
    rng = np.random.default_rng(d + 17 * kb + vb)
    cache, ref = new_cache(rng, 9, 2, d, 64, kb, vb)
    table = new_table(rng, 3, 3, 9)
    lengths, starts = np.array([37, 130, 5], np.int32), np.array([0, 37, 78, 80], np.int32)
    k, v = tokens(rng, 84, 2, d)                  # four rows of padding
    k[20, 1, 9], v[21, 0, 3], v[50, 1, 1] = np.inf, np.nan, -np.inf
    qlin.kv_write(cache, dev(k), dev(v), dev(table), dev(lengths), starts=dev(starts))
    store(ref, k, v, table, lengths, starts)
    got = host(cache.data).reshape(ref.data.shape)
    assert np.array_equal(got, ref.data)
    # one more token each
    lengths = lengths + 1
    k, v = tokens(rng, 3, 2, d)
    qlin.kv_write(cache, dev(k), dev(v), dev(table), dev(lengths))
    store(ref, k, v, table, lengths, None)
    assert np.array_equal(host(cache.data).reshape(ref.data.shape), ref.data)
    # and read back: all but the first tokens of each
    starts = np.array([0, 38, 150, 153], np.int32)
    for dtype, limit in ((torch.float32, 1e30), (torch.float16, 65504.0)):
        K = torch.full((156, 2, d), 7.0, dtype=dtype, device=DEV)
        V = torch.full((156, 2, d), 7.0, dtype=dtype, device=DEV)
        qlin.kv_read(cache, dev(table), dev(lengths), starts=dev(starts), K=K, V=V, dtype=dtype)
        for which, x, bits in ((0, host(K), kb), (1, host(V), vb)):
            want = np.full(x.shape, 7.0)
            for r, b, pos in kr.rows_of(lengths, starts, 156):
                want[r] = ref.get(*ref.token(table, b, pos), which)
            if bits < 16:
                want = np.clip(want, -limit, limit)
            assert np.array_equal(x, want.astype(x.dtype), equal_nan=True)


def test_values_next_to_the_largest():
    """Groups with fp16's largest values: the codes' values may lie beyond, the fp16 rows do not."""
    rng = np.random.default_rng(1)
    for bits in (4, 8):
        cache, ref = new_cache(rng, 2, 1, 64, 32, bits, bits)
        table, lengths = np.array([[1]], np.int32), np.array([8], np.int32)
        k = (65504 * rng.choice([-1, 1, 0.3, 0.999], (8, 1, 64))).astype(np.float16)
        starts = np.array([0, 8], np.int32)
        qlin.kv_write(cache, dev(k), dev(k), dev(table), dev(lengths), starts=dev(starts))
        store(ref, k, k, table, lengths, starts)
        assert np.array_equal(host(cache.data).reshape(ref.data.shape), ref.data)
        got = host(qlin.kv_read(cache, dev(table), dev(lengths), starts=dev(starts), rows=8)[0])
        want = np.clip([ref.get(1, i, 0) for i in range(8)], -65504, 65504).astype(np.float16)
        assert np.array_equal(got, want) and np.isfinite(got).all()


@pytest.mark.parametrize("seqs", [1, 70, 200])
def test_rows_of_many_sequences(seqs):
    """Ragged rows over more sequences than a wave has lanes, some without rows; tokens that are
    not there (a negative position, a page outside the cache, beyond the table) are left out and
    read as zeros."""
    rng = np.random.default_rng(seqs)
    pages = 3 * seqs + 1
    cache, ref = new_cache(rng, pages, 1, 64, 32, 8, 4)
    table = new_table(rng, seqs, 3, pages)
    table[rng.random(table.shape) < 0.1] = rng.choice([-1, pages, 2 ** 31 - 1, -2 ** 31])
    counts = rng.integers(0, 70, seqs)
    lengths = (counts + rng.integers(-20, 60, seqs)).astype(np.int32)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    m = int(starts[-1]) + 3
    k, v = tokens(rng, m, 1, 64)
    qlin.kv_write(cache, dev(k), dev(v), dev(table), dev(lengths), starts=dev(starts))
    store(ref, k, v, table, lengths, starts)
    assert np.array_equal(host(cache.data).reshape(ref.data.shape), ref.data)
    K = torch.full((m, 1, 64), 7.0, device=DEV)
    V = K.clone()
    qlin.kv_read(cache, dev(table), dev(lengths), starts=dev(starts), K=K, V=V, dtype=torch.float32)
    for which, x in ((0, host(K)), (1, host(V))):
        want = np.full((m, 1, 64), 7.0)
        for r, b, pos in kr.rows_of(lengths, starts, m):
            at = ref.token(table, b, pos)
            want[r] = 0 if at is None else ref.get(*at, which)
        assert np.array_equal(x, want.astype(np.float32))


def test_strided_rows():
    """Keys and values as parts of one projection's rows, and read into wider rows."""
    rng = np.random.default_rng(3)
    cache, ref = new_cache(rng, 6, 2, 64, 32, 4, 8)
    table, lengths = new_table(rng, 2, 3, 6), np.array([40, 9], np.int32)
    starts = np.array([0, 40, 49], np.int32)
    qkv = rng.standard_normal((49, 8, 64)).astype(np.float16)
    x = dev(qkv)
    qlin.kv_write(cache, x[:, 4:6], x[:, 6:], dev(table), dev(lengths), starts=dev(starts))
    store(ref, qkv[:, 4:6], qkv[:, 6:], table, lengths, starts)
    assert np.array_equal(host(cache.data).reshape(ref.data.shape), ref.data)
    out = torch.zeros(49, 8, 64, dtype=torch.float16, device=DEV)
    qlin.kv_read(cache, dev(table), dev(lengths), starts=dev(starts), K=out[:, :2], V=out[:, 5:7])
    got = host(out)
    dense = [host(t) for t in qlin.kv_read(cache, dev(table), dev(lengths), starts=dev(starts), rows=49)]
    assert np.array_equal(got[:, :2], dense[0]) and np.array_equal(got[:, 5:7], dense[1])
    assert not got[:, 2:5].any() and not got[:, 7:].any()


def attend(cache, ref, q, table, lengths, window=0, scale=None):
    o, o16, lse = qlin.kv_attention(cache, dev(q), dev(table), dev(lengths), window=window,
                                    scale=scale, want_lse=True)
    want, wl, eo, el = kr.attention(ref, q, table, lengths,
                                    cache.head_dim ** -0.5 if scale is None else scale, window)
    o, o16, lse = host(o), host(o16), host(lse)
    kr.check(o, want, eo, "O")
    kr.check16(o16, want, eo, "O16")
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), empty) and not o[empty].any() and not o16[empty].any()
    kr.check(lse[~empty], wl[~empty], el[~empty], "lse")
    return o


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kb,vb", BITS)
def test_attention(d, kb, vb):
    rng = np.random.default_rng(1000 + d + 17 * kb + vb)
    lengths = np.array([0, 1, 31, 32, 33, 200, 64, -5], np.int32)
    heads, ratio = 2, 3
    cache, ref = new_cache(rng, 60, heads, d, 32, kb, vb)
    table = new_table(rng, 8, 7, 60)
    fill(rng, cache, ref, table, lengths)
    q = (1.5 * rng.standard_normal((8, heads * ratio, d))).astype(np.float16)
    for window in (0, 1, 40):
        attend(cache, ref, q, table, lengths, window)


@pytest.mark.parametrize("ratio", [1, 2, 7, 16, 17, 40])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
def test_attention_heads_and_pages(ratio, page):
    rng = np.random.default_rng(ratio * page)
    lengths = np.array([300, 17, 513], np.int32)
    width = -(-600 // page)
    cache, ref = new_cache(rng, 3 * width + 2, 1, 64, page, 4, 4)
    table = new_table(rng, 3, width, 3 * width + 2)
    fill(rng, cache, ref, table, lengths)
    q = rng.standard_normal((3, ratio, 64)).astype(np.float16)
    attend(cache, ref, q, table, lengths, window=page + 3 if ratio % 2 else 0)


def test_attention_bad_pages_and_lengths():
    """Pages outside the cache and lengths beyond the table: those tokens are not there."""
    rng = np.random.default_rng(5)
    lengths = np.array([200, 200, 100, 96, 2 ** 31 - 1, 150], np.int32)
    cache, ref = new_cache(rng, 40, 2, 64, 32, 8, 8)
    table = new_table(rng, 6, 6, 40)
    fill(rng, cache, ref, table, np.full(6, 192, np.int32))
    table[0, 2], table[1, :], table[2, 3], table[3, 0], table[5, 4] = -1, -7, 40, 2 ** 31 - 1, -2 ** 31
    q = rng.standard_normal((6, 4, 64)).astype(np.float16)
    for window in (0, 33):
        inside = np.minimum(lengths, 192) if window == 0 else lengths
        ref_lengths = np.array([min(int(n), 400) for n in inside], np.int32) if window else inside
        if window:      # a window behind the table's end sees nothing
            ref_lengths[4] = 400
        o, _, lse = qlin.kv_attention(cache, dev(q), dev(table), dev(lengths), window=window,
                                      want_lse=True)
        want, wl, eo, el = kr.attention(ref, q, table, ref_lengths, 64 ** -0.5, window)
        kr.check(host(o), want, eo, "O")
        assert np.array_equal(np.isneginf(host(lse)), np.isneginf(wl))


@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (16, 16)])
def test_attention_ignores_what_is_not_seen(kb, vb):
    """Behind the end, before the window and in other pages anything may lie, NaN included."""
    rng = np.random.default_rng(6)
    lengths = np.array([45, 70, 3], np.int32)
    cache, ref = new_cache(rng, 12, 1, 128, 32, kb, vb)
    table = new_table(rng, 3, 3, 12)
    fill(rng, cache, ref, table, np.full(3, 96, np.int32))
    q = rng.standard_normal((3, 5, 128)).astype(np.float16)
    clean = attend(cache, ref, q, table, lengths, 20)
    nan = np.full((1, 128), np.nan, np.float16)
    for page in range(12):
        for at in range(32):
            owner = np.argwhere(table == page)
            if len(owner):
                pos = owner[0, 1] * 32 + at
                n = lengths[owner[0, 0]]
                if max(n - 20, 0) <= pos < n:
                    continue
            ref.put(page, at, 0, 0, nan[0])
            ref.put(page, at, 0, 1, nan[0])
    cache.data.copy_(dev(ref.data.reshape(tuple(cache.data.shape))))
    o = host(qlin.kv_attention(cache, dev(q), dev(table), dev(lengths), window=20)[0])
    assert np.array_equal(o, clean)
    # a NaN among the seen tokens of sequence 0 stays in its row
    ref.put(table[0, 1], 3, 0, 0, nan[0])
    cache.data.copy_(dev(ref.data.reshape(tuple(cache.data.shape))))
    o = host(qlin.kv_attention(cache, dev(q), dev(table), dev(lengths), window=20)[0])
    assert np.isnan(o[0]).all() and np.array_equal(o[1:], clean[1:])


@pytest.mark.parametrize("vb", [4, 8, 16])
@pytest.mark.parametrize("size", [6e-8, 1e-4, 1.0, 3e4])
def test_attention_sizes_of_values(vb, size):
    """Values of any size keep their bits, and scores far apart: one token with most of the weight,
    a thousand with little."""
    rng = np.random.default_rng(7)
    n = 1000
    cache, ref = new_cache(rng, 32, 1, 64, 32, 16, vb)
    table = new_table(rng, 1, 32, 32)
    k = 0.1 * rng.standard_normal((n, 1, 64))
    k[500, 0] = 1.0
    k[100:400, 0, :8] -= 0.5
    v = (size * rng.uniform(-2, 2, (n, 1, 64)) * rng.choice([1.0, 0.01], (n, 1, 1))).astype(np.float16)
    lengths, starts = np.array([n], np.int32), np.array([0, n], np.int32)
    qlin.kv_write(cache, dev(k.astype(np.float16)), dev(v), dev(table), dev(lengths), starts=dev(starts))
    ref.data[:] = host(cache.data).reshape(ref.data.shape)
    q = np.stack([np.full((1, 64), c) for c in (0.1, 1.0, 2.0)], 1).astype(np.float16)
    attend(cache, ref, q, table, lengths)


def test_attention_split_over_a_long_sequence():
    """Sequences dealt out over all work-groups and joined, beside short ones; the same twice."""
    rng = np.random.default_rng(8)
    lengths = np.array([6000, 1, 0, 2500, 33, 700], np.int32)
    cache, ref = new_cache(rng, 6 * 48, 2, 64, 128, 8, 8)
    table = new_table(rng, 6, 48, 6 * 48)
    fill(rng, cache, ref, table, lengths)
    q = rng.standard_normal((6, 4, 64)).astype(np.float16)
    first = attend(cache, ref, q, table, lengths)
    assert np.array_equal(first, attend(cache, ref, q, table, lengths))
    attend(cache, ref, q, table, lengths, window=3001)


@pytest.mark.parametrize("seqs", [65, 300])
def test_attention_of_many_sequences(seqs):
    rng = np.random.default_rng(seqs)
    lengths = rng.integers(0, 60, seqs).astype(np.int32)
    cache, ref = new_cache(rng, 2 * seqs, 1, 64, 32, 8, 4)
    table = new_table(rng, seqs, 2, 2 * seqs)
    fill(rng, cache, ref, table, lengths)
    q = rng.standard_normal((seqs, 2, 64)).astype(np.float16)
    attend(cache, ref, q, table, lengths)


def test_attention_strided_and_given_outputs():
    rng = np.random.default_rng(9)
    lengths = np.array([50, 90], np.int32)
    cache, ref = new_cache(rng, 6, 2, 64, 32, 4, 4)
    table = new_table(rng, 2, 3, 6)
    fill(rng, cache, ref, table, lengths)
    qkv = dev(rng.standard_normal((2, 8, 64)).astype(np.float16))
    want = qlin.kv_attention(cache, qkv[:, :4].contiguous(), dev(table), dev(lengths), want_lse=True)
    O = torch.full((2, 6, 64), 3.0, device=DEV)
    O16 = torch.full((2, 6, 64), 3.0, dtype=torch.float16, device=DEV)
    wide = dev(np.concatenate([table, table[:, :1] * 0 - 1], 1))[:, :3]
    qlin.kv_attention(cache, qkv[:, :4], wide, dev(lengths), O=O[:, :4], O16=O16[:, :4])
    torch.cuda.synchronize()
    assert torch.equal(O[:, :4], want[0]) and torch.equal(O16[:, :4], want[1])
    assert (O[:, 4:] == 3).all() and (O16[:, 4:] == 3).all()
    alone = qlin.kv_attention(cache, qkv[:, :4], dev(table), dev(lengths), want_o=False)
    assert alone[0] is None and alone[2] is None and torch.equal(alone[1], want[1])


def test_cache_of_more_than_4_gib():
    """Pages whose bytes lie beyond 32 bits."""
    rng = np.random.default_rng(10)
    size = qlin.kv_page_bytes(128, 256, 16, 16)
    pages = 5 * 2 ** 30 // size // 2 + 1
    cache = qlin.kv_cache(pages, 2, 128, 256, 16, 16)
    small, ref = new_cache(rng, 4, 2, 128, 256, 16, 16)
    lengths, starts = np.array([300, 10], np.int32), np.array([0, 300, 310], np.int32)
    table = np.array([[1, 3], [2, 0]], np.int32)
    far = np.array([[pages - 1, 5], [pages // 2, 7]], np.int32)
    k, v = tokens(rng, 310, 2, 128)
    q = rng.standard_normal((2, 4, 128)).astype(np.float16)
    out = []
    for c, t in ((small, table), (cache, far)):
        qlin.kv_write(c, dev(k), dev(v), dev(t), dev(lengths), starts=dev(starts))
        out.append([host(x) for x in (*qlin.kv_read(c, dev(t), dev(lengths), starts=dev(starts), rows=310),
                                      *qlin.kv_attention(c, dev(q), dev(t), dev(lengths))[:2])])
    assert all(np.array_equal(a, b) for a, b in zip(*out))
    assert np.array_equal(out[0][0], k) and np.array_equal(out[0][1], v)


def test_decode_steps_in_a_graph():
    """Steps as they are used: each sequence's new token goes into the cache and attends, recorded
    once and replayed on longer and longer sequences, with other calls in between."""
    rng = np.random.default_rng(11)
    heads, d, seqs = 2, 64, 3
    cache, ref = new_cache(rng, 12, heads, d, 32, 8, 4)
    table = new_table(rng, seqs, 4, 12)
    lengths = np.array([30, 1, 63], np.int32)
    fill(rng, cache, ref, table, lengths)
    k, v = (torch.zeros(seqs, heads, d, dtype=torch.float16, device=DEV) for _ in range(2))
    q = torch.zeros(seqs, 6, d, dtype=torch.float16, device=DEV)
    dl, dt = dev(lengths), dev(table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):               # (first use, outside the graph)
        qlin.kv_attention(cache, q, dt, dl)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dl.add_(1)
        qlin.kv_write(cache, k, v, dt, dl)
        o, o16, lse = qlin.kv_attention(cache, q, dt, dl, want_lse=True)
    for step in range(5):
        lengths = lengths + 1
        kn, vn = tokens(rng, seqs, heads, d)
        kn = np.clip(kn, -8, 8)
        qn = rng.standard_normal((seqs, 6, d)).astype(np.float16)
        for t, x in ((k, kn), (v, vn), (q, qn)):
            t.copy_(dev(x))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
            again = qlin.kv_attention(cache, q, dt, dl)[0]
        torch.cuda.synchronize()
        store(ref, kn, vn, table, lengths, None)
        assert np.array_equal(host(cache.data).reshape(ref.data.shape), ref.data)
        want, wl, eo, el = kr.attention(ref, qn, table, lengths, d ** -0.5, 0)
        kr.check(host(o), want, eo, "O")
        kr.check(host(lse), wl, el, "lse")
        assert torch.equal(o, again)


def test_two_graphs_and_streams():
    """Two recorded calls replayed at the same time on two streams do not share scratch memory."""
    rng = np.random.default_rng(12)
    cache, ref = new_cache(rng, 100, 2, 64, 128, 4, 4)
    table = new_table(rng, 2, 50, 100)
    lengths = np.array([6000, 5000], np.int32)
    fill(rng, cache, ref, table, lengths)
    dt, dl = dev(table), dev(lengths)
    qs = [dev(rng.standard_normal((2, 4, 64)).astype(np.float16)) for _ in range(2)]
    want = [qlin.kv_attention(cache, q, dt, dl)[0].clone() for q in qs]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for q, s in zip(qs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(qlin.kv_attention(cache, q, dt, dl)[0])
        graphs.append(graph)
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
                graph.replay()
        eager = [qlin.kv_attention(cache, q, dt, dl)[0] for q in qs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(e, b) for a, b, e in zip(outs, want, eager))
