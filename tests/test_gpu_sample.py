"""Drawing tokens on a GPU against the 64-bit reference of tests/sample_ref.py."""
import numpy as np
import pytest
import torch

import sample_ref as sr
from group_wise_bit_amd import qlin

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN, BIG = np.inf, np.nan, float(np.finfo(np.float32).max)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def arrays(temperature=None, top_k=None, top_p=None, min_p=None):
    return [None if v is None else np.asarray(v, d)
            for v, d in ((temperature, np.float32), (top_k, np.int32), (top_p, np.float32),
                         (min_p, np.float32))]


def draw(logits, u, *settings):
    s = qlin.Sampling(*[None if v is None else dev(v) for v in settings])
    ids, probs = qlin.sample(s, dev(logits), dev(u))
    return host(ids), host(probs)


def run(logits, u, what, **kw):
    s = arrays(**kw)
    ids, probs = draw(logits, u, *s)
    sr.check(ids, probs, sr.sample(logits, u, *s), what)
    return ids, probs


def logits_of(rng, m, vocab, std=2.0, rounded=False):
    x = std * rng.standard_normal((m, vocab))
    x += (rng.random((m, vocab)) < 1e-3) * rng.uniform(0, 5, (m, vocab))
    return x.astype(np.float16 if rounded else np.float32).astype(np.float32)


@pytest.mark.parametrize("vocab", [1, 2, 7, 64, 255, 1000, 1025, 4097, 32003, 151936, 262144])
@pytest.mark.parametrize("rounded", [False, True])
def test_settings(vocab, rounded):
    """Every setting alone and with the others, over ordinary logits and ones with many ties."""
    rng = np.random.default_rng(vocab + rounded)
    m = 12 if vocab < 100000 else 5
    logits = logits_of(rng, m, vocab, rounded=rounded)
    u = rng.random(m).astype(np.float32)
    t = rng.choice([0.5, 0.7, 1.0, 1.3], m)
    k = rng.choice([1, 2, 5, 40, 300, 5000, 10 ** 6, 0, -3], m)
    p = rng.choice([0.1, 0.5, 0.9, 0.99, 1.0], m)
    mp = rng.choice([0.0, 0.001, 0.05, 0.3], m)
    run(logits, u, "plain")
    run(logits, u, "temperature", temperature=t)
    run(logits, u, "top_k", temperature=t, top_k=k)
    run(logits, u, "top_p", temperature=t, top_p=p)
    run(logits, u, "min_p", temperature=t, min_p=mp)
    run(logits, u, "all", temperature=t, top_k=k, top_p=p, min_p=mp)


def test_greedy():
    rng = np.random.default_rng(1)
    logits = logits_of(rng, 9, 5000, rounded=True)
    u = rng.random(9).astype(np.float32)
    for kw in (dict(temperature=np.zeros(9)), dict(temperature=[-1, 0, NAN, -INF, 0, 0, 0, 0, 0]),
               dict(top_k=np.ones(9)), dict(top_p=np.zeros(9)), dict(top_p=np.full(9, -1.0))):
        ids, probs = draw(logits, u, *arrays(**kw))
        assert np.array_equal(ids, logits.argmax(1)) and (probs == 1).all(), kw


@pytest.mark.parametrize("vocab", [8, 4096, 65536])
def test_ties_and_borders(vocab):
    """Equal logits: every sum is exact, and a border falls to the next token."""
    logits = np.zeros((8, vocab), np.float32)
    u = (np.arange(8) / 8).astype(np.float32)
    step = vocab // 8
    ids, probs = draw(logits, u, None, None, None, None)
    assert np.array_equal(ids, np.arange(8) * step) and np.allclose(probs, 1 / vocab, rtol=1e-7)
    below = np.nextafter(u[1:], np.float32(0))
    ids, _ = draw(logits[1:], below, None, None, None, None)
    assert np.array_equal(ids, np.arange(1, 8) * step - 1)
    # the first k by index; half of the mass is half of the tokens
    k = np.maximum(np.arange(8) * step // 2, 1).astype(np.int32)
    last = np.full(8, np.nextafter(np.float32(1), np.float32(0)))
    ids, _ = draw(logits, last, None, k, None, None)
    assert np.array_equal(ids, k - 1)
    ids, _ = draw(logits, last, None, None, np.full(8, 0.5, np.float32), None)
    assert (ids == vocab // 2 - 1).all()
    ids, _ = draw(logits, last, None, None, None, np.ones(8, np.float32))
    assert (ids == vocab - 1).all()


def test_random_numbers_out_of_range():
    rng = np.random.default_rng(2)
    logits = logits_of(rng, 6, 3001)
    first = [sr.kept_tokens(r, 1, 50, 1, 0)[0].min() for r in logits]
    last = [sr.kept_tokens(r, 1, 50, 1, 0)[0].max() for r in logits]
    k = np.full(6, 50, np.int32)
    for v, want in ((0.0, first), (-0.5, first), (NAN, first), (-INF, first), (1.0, last), (7.0, last),
                    (INF, last)):
        ids, _ = draw(logits, np.full(6, v, np.float32), None, k, None, None)
        assert np.array_equal(ids, want), v


def test_masked_tokens():
    """-inf and NaN are no tokens, +inf is the largest number, the type's lowest value a token
    without weight; rows without tokens."""
    rng = np.random.default_rng(3)
    logits = logits_of(rng, 10, 2000)
    logits[0, rng.random(2000) < 0.7] = -INF
    logits[1, rng.random(2000) < 0.7] = NAN
    logits[2, rng.random(2000) < 0.7] = -BIG
    logits[3] = -INF
    logits[4] = NAN
    logits[5, [7, 900]] = INF
    logits[6] = -BIG
    logits[7] = -INF
    logits[7, 1999] = -BIG
    logits[8, :] = -INF
    logits[8, [3, 5]] = [1.0, 2.0]
    logits[9] = INF
    u = rng.random(10).astype(np.float32)
    for kw in (dict(), dict(top_k=np.full(10, 30)), dict(top_p=np.full(10, 0.9)),
               dict(min_p=np.full(10, 0.01)), dict(temperature=np.full(10, 0.6), top_k=np.full(10, 1500),
                                                   top_p=np.full(10, 0.8))):
        ids, probs = run(logits, u, kw, **kw)
        assert (ids[3:5] == -1).all() and (probs[3:5] == 0).all() and ids[7] == 1999


@pytest.mark.parametrize("t", [1e-30, 1e-6, 0.02, 20.0, 1e4, 3e38, INF])
def test_temperatures_far_out(t):
    """Nearly greedy, and nearly uniform over the whole row."""
    rng = np.random.default_rng(4)
    logits = logits_of(rng, 6, 20011)
    u = rng.random(6).astype(np.float32)
    kw = dict(temperature=np.full(6, t))
    run(logits, u, "plain", **kw)
    run(logits, u, "top_k", top_k=[3, 50, 1000, 5000, 19999, 0], **kw)
    run(logits, u, "top_p", top_p=[0.013, 0.3, 0.53, 0.91, 0.999, 1.0], **kw)
    run(logits, u, "all", top_k=[3, 50, 1000, 5000, 19999, 0], top_p=[0.013, 0.3, 0.53, 0.91, 0.999, 1.0],
        min_p=[0.0, 0.9, 0.0, 0.9999, 0.5, 0.1], **kw)


def test_many_rows_and_strides():
    rng = np.random.default_rng(5)
    wide = dev(logits_of(rng, 700, 1500))
    logits = wide[:, 100:1111]
    u = rng.random(700).astype(np.float32)
    s = arrays(temperature=rng.uniform(0.3, 1.5, 700), top_k=rng.integers(0, 100, 700),
               top_p=rng.uniform(0.3, 1.1, 700), min_p=rng.uniform(0, 0.1, 700))
    ids, probs = qlin.sample(qlin.Sampling(*map(dev, s)), logits, dev(u))
    ref = sr.sample(host(logits), u, *s)
    sr.check(host(ids), host(probs), ref, "strided")
    out = torch.full((700,), -7, dtype=torch.int32, device=DEV)
    assert qlin.sample(qlin.Sampling(*map(dev, s)), logits, dev(u), ids=out)[0] is out
    assert torch.equal(out, ids)
    one = qlin.sample(qlin.Sampling(), wide[3:4, 5:8], dev(u[:1]))[0]
    assert host(one)[0] == sr.sample(host(wide[3:4, 5:8]), u[:1])[0][0]


def test_draws_follow_the_probabilities():
    """Evenly spread u on one row: every kept token comes up as often as its probability says."""
    rng = np.random.default_rng(6)
    row = logits_of(rng, 1, 50)[0]
    n = 4096
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    ids, _ = draw(np.tile(row, (n, 1)), u, np.full(n, 0.8, np.float32), np.full(n, 20, np.int32),
                  None, None)
    order, mass, _ = sr.kept_tokens(row, 0.8, 20, 1.0, 0.0)
    want = np.zeros(50)
    want[order] = mass / mass.sum()
    assert np.abs(np.bincount(ids, minlength=50) / n - want).max() <= 1.0 / n + 1e-6


def test_graph_and_streams():
    """Recorded once, replayed with new logits and random numbers, eager calls in between; two
    graphs at the same time."""
    rng = np.random.default_rng(7)
    m, vocab = 6, 40000
    s = arrays(temperature=np.full(m, 0.8), top_k=np.full(m, 200), top_p=np.full(m, 0.9))
    sampling = qlin.Sampling(*[None if v is None else dev(v) for v in s])
    ins = [(torch.zeros(m, vocab, device=DEV), torch.zeros(m, device=DEV)) for _ in range(2)]
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for (x, u), stream in zip(ins, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(qlin.sample(sampling, x, u))
        graphs.append(graph)
    for step in range(4):
        given = []
        for x, u in ins:
            lx, lu = logits_of(rng, m, vocab), rng.random(m).astype(np.float32)
            x.copy_(dev(lx))
            u.copy_(dev(lu))
            given.append((lx, lu))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = [qlin.sample(sampling, x, u) for x, u in ins]
        torch.cuda.synchronize()
        for (lx, lu), (ids, probs), e in zip(given, outs, eager):
            sr.check(host(ids), host(probs), sr.sample(lx, lu, *s), step)
            assert torch.equal(ids, e[0]) and torch.equal(probs, e[1])


def test_from_the_lm_head():
    """As it is used: logits of a decode batch from the packed LM head, then the draw."""
    rng = np.random.default_rng(8)
    w = qlin.quantize(dev((0.02 * rng.standard_normal((5000, 256))).astype(np.float16)), 8, 64)
    x = dev((4 * rng.standard_normal((7, 256))).astype(np.float16))
    logits = qlin.gemm(w, x)
    u = rng.random(7).astype(np.float32)
    s = arrays(temperature=np.full(7, 0.3), top_p=np.full(7, 0.9))
    ids, probs = qlin.sample(qlin.Sampling(*[None if v is None else dev(v) for v in s]), logits, dev(u))
    sr.check(host(ids), host(probs), sr.sample(host(logits), u, *s), "head")
    # and the embedding of the drawn tokens
    row = host(qlin.embed_rows(w, ids)[0])
    assert row.shape == (7, 256)
