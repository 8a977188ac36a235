"""The cache of keys and values on a GPU where it is easy to go wrong: scales of every sign, pages
that sequences share, work-groups whose tiles lie in many pages, other streams and threads, the
largest and smallest batches, steps from the projections to the output's."""
import threading

import numpy as np
import pytest
import torch

import kv_ref as kr
from group_wise_bit_amd import qlin
from test_gpu_kv import attend, dev, fill, host, new_cache, new_table, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scale", [-0.125, -1.0, 0.0, 1e-40, 1e-6, 3.0])
def test_scales(scale):
    """Negative scales turn the scores round; with 0 every token weighs the same."""
    rng = np.random.default_rng(1)
    lengths = np.array([0, 1, 70, 200], np.int32)
    cache, ref = new_cache(rng, 28, 2, 64, 32, 8, 4)
    table = new_table(rng, 4, 7, 28)
    fill(rng, cache, ref, table, lengths)
    q = rng.standard_normal((4, 4, 64)).astype(np.float16)
    for window in (0, 33):
        o = qlin.kv_attention(cache, dev(q), dev(table), dev(lengths), scale=scale, window=window,
                              want_lse=True)
        want, wl, eo, el = kr.attention(ref, q, table, lengths, np.float32(scale).astype(float), window)
        kr.check(host(o[0]), want, eo, "O")
        seen = ~np.isneginf(wl)
        kr.check(host(o[2])[seen], wl[seen], el[seen], "lse")


def test_shared_pages():
    """Sequences with one prefix read its pages together, a page stands in a row twice, and what
    one of them writes behind it does not show in the others."""
    rng = np.random.default_rng(2)
    cache, ref = new_cache(rng, 12, 2, 128, 32, 4, 8)
    table = np.array([[5, 3, 0, 1], [5, 3, 2, 4], [5, 3, 6, 7], [5, 5, 3, 8]], np.int32)
    first = np.array([64], np.int32)
    fill(rng, cache, ref, table[:1], first)                    # the prefix
    lengths = np.array([70, 90, 65, 99], np.int32)
    counts = np.array([6, 26, 1, 3])
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    k, v = tokens(rng, int(starts[-1]), 2, 128)
    k = np.clip(k, -8, 8).astype(np.float16)
    qlin.kv_write(cache, dev(k), dev(v), dev(table), dev(lengths), starts=dev(starts))
    for r, b, pos in kr.rows_of(lengths, starts, len(k)):
        for h in range(2):
            ref.put(*ref.token(table, b, pos), h, 0, k[r, h])
            ref.put(*ref.token(table, b, pos), h, 1, v[r, h])
    assert np.array_equal(host(cache.data).reshape(ref.data.shape), ref.data)
    q = rng.standard_normal((4, 6, 128)).astype(np.float16)
    attend(cache, ref, q, table, lengths)


@pytest.mark.parametrize("kb,vb", [(4, 4), (16, 16)])
def test_tiles_in_many_pages(kb, vb):
    """The same memory as pages of 256 and of 32 tokens gives the same bits, also where a
    work-group's tiles lie in more pages than a wave has lanes."""
    rng = np.random.default_rng(3)
    length = 1024 * 32 * 80 if kb == 4 else 256 * 32 * 300
    pages = -(-length // 256)
    big = qlin.kv_cache(pages, 1, 64, 256, kb, vb)
    big.data.view(torch.int32)[:] = torch.randint(-2 ** 31, 2 ** 31 - 1, big.data.view(torch.int32).shape,
                                                  dtype=torch.int32, device=DEV)
    if kb == 16:
        v = big.data.view(torch.float16)
        torch.nan_to_num(v, 0, 0, 0, out=v)
        v.clamp_(-4, 4)
    else:                                       # scales: positive, from 2^-8 to 2
        tile = big.data.view(pages, 8, -1)
        s = tile[:, :, 2048:2176].contiguous().view(torch.int16)
        tile[:, :, 2048:2176] = ((s & 0x1FFF) + 0x1C00).view(torch.uint8).reshape(pages, 8, 128)
    small = qlin.KVCache(big.data.view(pages * 8, 1, -1), 1, 64, 32, kb, vb)
    table = torch.randperm(pages, device=DEV).to(torch.int32)[None].contiguous()
    fine = (table[:, :, None] * 8 + torch.arange(8, dtype=torch.int32, device=DEV)).view(1, -1)
    lengths = torch.tensor([length - 5], dtype=torch.int32, device=DEV)
    q = torch.randn(1, 4, 64, device=DEV).half()
    a = qlin.kv_attention(big, q, table, lengths, want_lse=True)
    b = qlin.kv_attention(small, q, fine, lengths, want_lse=True)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.isfinite(a[0]).all() and a[0].abs().max() > 0
    # half of it against the other half and the log-sum-exp's join: a sequence split by the caller
    half = pages // 2
    parts = [qlin.kv_attention(big, q, t.contiguous(), l, want_lse=True) for t, l in (
        (table[:, :half], torch.tensor([half * 256], dtype=torch.int32, device=DEV)),
        (table[:, half:], lengths - half * 256))]
    w = torch.softmax(torch.stack([p[2].double() for p in parts]), 0)
    joined = sum(w[i][..., None] * parts[i][0].double() for i in range(2))
    assert (joined - a[0].double()).abs().max() <= 1e-4 * a[0].abs().max()


def test_whole_and_split_agree():
    """The same sequences under a table just short enough not to be split, and a longer one."""
    rng = np.random.default_rng(4)
    lengths = np.array([1000, 3, 0, 512, 1024], np.int32)
    cache, ref = new_cache(rng, 5 * 32, 1, 128, 32, 8, 8)
    table = new_table(rng, 5, 32, 5 * 32)
    fill(rng, cache, ref, table, lengths)
    q = rng.standard_normal((5, 20, 128)).astype(np.float16)
    attend(cache, ref, q, table, lengths)
    attend(cache, ref, q, np.concatenate([table, -np.ones((5, 1), np.int32)], 1), lengths)


def test_threads_and_streams():
    """Threads on one stream, and a call on another stream than the tensors were made on."""
    rng = np.random.default_rng(5)
    cache, ref = new_cache(rng, 100, 2, 64, 64, 4, 4)
    table = new_table(rng, 2, 50, 100)
    lengths = np.array([3000, 1500], np.int32)
    fill(rng, cache, ref, table, lengths)
    dt, dl = dev(table), dev(lengths)
    qs = [dev(rng.standard_normal((2, 2 * r, 64)).astype(np.float16)) for r in (1, 3, 8, 20)]
    want = [qlin.kv_attention(cache, q, dt, dl)[0] for q in qs]
    logits = [torch.randn(m, 9000, device=DEV) for m in (1, 5, 40, 3)]
    us = [torch.rand(len(x), device=DEV) for x in logits]
    ids = [qlin.sample(qlin.Sampling(), x, u)[0] for x, u in zip(logits, us)]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def run(i):
        for _ in range(20):
            got[i].append((qlin.kv_attention(cache, qs[i], dt, dl)[0],
                           qlin.sample(qlin.Sampling(), logits[i], us[i])[0]))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(4):
        assert len(got[i]) == 20
        assert all(torch.equal(o, want[i]) and torch.equal(d, ids[i]) for o, d in got[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = qlin.kv_attention(cache, qs[1], dt, dl)[0]
    side.synchronize()
    assert torch.equal(o, want[1])


def test_empty_batches():
    cache = qlin.kv_cache(2, 2, 64, 32, 4, 4)
    none = torch.zeros(0, 2, 64, dtype=torch.float16, device=DEV)
    table, lengths = torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.zeros(
        0, dtype=torch.int32, device=DEV)
    qlin.kv_write(cache, none, none, table, lengths)
    assert qlin.kv_read(cache, table, lengths)[0].shape == (0, 2, 64)
    assert qlin.kv_attention(cache, none, table, lengths)[0].shape == (0, 2, 64)
    # sequences without rows
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    starts = torch.zeros(2, dtype=torch.int32, device=DEV)
    before = cache.data.clone()
    x = torch.randn(4, 2, 64, device=DEV).half()
    qlin.kv_write(cache, x, x, one[None], one, starts=starts)
    K = torch.full((4, 2, 64), 5.0, dtype=torch.float16, device=DEV)
    V = K.clone()
    qlin.kv_read(cache, one[None], one, starts=starts, K=K, V=V)
    torch.cuda.synchronize()
    assert torch.equal(cache.data, before) and (K == 5).all() and (V == 5).all()
    ids, probs = qlin.sample(qlin.Sampling(), torch.zeros(0, 9, device=DEV), torch.zeros(0, device=DEV))
    assert ids.shape == (0,) and probs.shape == (0,)


def test_workspace_given_and_too_small():
    rng = np.random.default_rng(6)
    cache, ref = new_cache(rng, 100, 2, 64, 64, 4, 4)
    table = new_table(rng, 2, 50, 100)
    lengths = np.array([3000, 1500], np.int32)
    fill(rng, cache, ref, table, lengths)
    q = dev(rng.standard_normal((2, 4, 64)).astype(np.float16))
    want = qlin.kv_attention(cache, q, dev(table), dev(lengths))[0]
    ws = torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV)
    got = qlin.kv_attention(cache, q, dev(table), dev(lengths), ws=ws)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (ws[:65536] == 255).all()
    for bad in (None, ws[:70000]):
        with pytest.raises(qlin.QlinError) as e:
            qlin.kv_attention(cache, q, dev(table), dev(lengths), ws=bad)
        assert e.value.status == 8
    x, u = torch.randn(3, 5000, device=DEV), torch.rand(3, device=DEV)
    assert torch.equal(qlin.sample(qlin.Sampling(), x, u, ws=ws)[0], qlin.sample(qlin.Sampling(), x, u)[0])
    assert (ws[:65536] == 255).all()
    with pytest.raises(qlin.QlinError):
        qlin.sample(qlin.Sampling(), x, u, ws=ws[:70000])


def test_a_decode_step():
    """As it is used: q, k and v of a batch from packed projections, the new tokens into the cache,
    attention, the output projection, the LM head, the draw and the next embedding."""
    rng = np.random.default_rng(7)
    heads, kvh, d, model, vocab, seqs = 14, 2, 64, 896, 3001, 5

    def weight(n, k, bits=4):
        return qlin.quantize(dev((0.03 * rng.standard_normal((n, k))).astype(np.float16)), bits, 64)
    wq, wk, wv = weight(heads * d, model), weight(kvh * d, model), weight(kvh * d, model)
    wo, head = weight(model, heads * d), weight(vocab, model, 8)
    cache, ref = new_cache(rng, 20, kvh, d, 32, 8, 8)
    table = new_table(rng, seqs, 4, 20)
    lengths = np.array([5, 64, 33, 1, 90], np.int32)
    fill(rng, cache, ref, table, lengths)
    x = dev(rng.standard_normal((seqs, model)).astype(np.float16))
    dl, dt = dev(lengths), dev(table)
    for _ in range(2):
        lengths, dl = lengths + 1, dl + 1
        q, k, v = (t.half() for t in qlin.gemm_multi([wq, wk, wv], x))
        q, k, v = q.view(seqs, heads, d), k.view(seqs, kvh, d), v.view(seqs, kvh, d)
        qlin.kv_write(cache, k, v, dt, dl)
        for b in range(seqs):
            at = ref.token(table, b, int(lengths[b]) - 1)
            for h in range(kvh):
                ref.put(*at, h, 0, host(k)[b, h])
                ref.put(*at, h, 1, host(v)[b, h])
        assert np.array_equal(host(cache.data).reshape(ref.data.shape), ref.data)
        o, o16, _ = qlin.kv_attention(cache, q, dt, dl)
        want, _, eo, _ = kr.attention(ref, host(q), table, lengths, d ** -0.5, 0)
        kr.check(host(o), want, eo, "O")
        y = qlin.gemm(wo, o16.view(seqs, heads * d))
        ids, probs = qlin.sample(qlin.Sampling(temperature=torch.full((seqs,), 0.7, device=DEV)),
                                 qlin.gemm(head, y.half()), torch.rand(seqs, device=DEV))
        torch.cuda.synchronize()
        assert ((ids >= 0) & (ids < vocab)).all() and (probs > 0).all()
        x = qlin.embed_rows(head, ids)[0]


@pytest.mark.parametrize("heads,kv_heads", [(1024, 256), (1024, 1), (513, 27), (256, 256)])
@pytest.mark.parametrize("width", [2, 40])
def test_many_heads(heads, kv_heads, width):
    """The most heads, few and many to a head of the cache, unsplit and split."""
    rng = np.random.default_rng(8)
    lengths = np.array([1, 45, 64], np.int32)
    cache, ref = new_cache(rng, 7, kv_heads, 64, 32, 4, 8)
    table = np.full((3, width), -1, np.int32)
    table[:, :2] = new_table(rng, 3, 2, 7)
    # (one head's tokens in all heads, each times its own power of two: the bytes are written by the call)
    k, v = tokens(rng, int(lengths.sum()), 1, 64)
    size = 2.0 ** rng.integers(-2, 3, (1, kv_heads, 1))
    k, v = (np.clip(x * size, -8, 8).astype(np.float16) for x in (k, v))
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    qlin.kv_write(cache, dev(k), dev(v), dev(table), dev(lengths), starts=dev(starts))
    ref.data[:] = host(cache.data).reshape(ref.data.shape)
    q = rng.standard_normal((3, heads, 64)).astype(np.float16)
    attend(cache, ref, q, table, lengths)
