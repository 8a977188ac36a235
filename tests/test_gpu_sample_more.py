"""Drawing tokens on a GPU: settings out of range among ties, rows in many batches, long flat rows,
rows whose cuts lie far apart, draws that other rows do not change."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import sample_ref as sr
from group_wise_bit_amd import qlin
from test_gpu_sample import BIG, DEV, INF, NAN, arrays, draw, host, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [5, 700, 9000, 40000])
def test_min_p_above_one_among_ties(vocab):
    """With min_p 1 every token of the largest logit is kept, above it the first alone."""
    x = np.zeros((6, vocab), np.float32)
    x[:, 3:] = -1
    x[:, [vocab - 1, vocab // 2]] = 2
    for mp in (1.0, 1.0000001, 1.5, 3e38, INF):
        u = np.array([0, .25, .49, .51, .75, .9999], np.float32)
        # (p = exp(0) is exactly 1, so that min_p 1 is no border that a rounding could cross)
        ids, probs = draw(x, u, *arrays(min_p=[mp] * 6))
        if mp > 1:
            assert (ids == vocab // 2).all() and (probs == 1).all()
        else:
            assert ids.tolist() == [vocab // 2] * 3 + [vocab - 1] * 3 and (probs == .5).all()


def test_settings_that_are_no_numbers():
    """NaN is off, except for the temperature (not above 0)."""
    rng = np.random.default_rng(1)
    x = (3 * rng.standard_normal((4, 20000))).astype(np.float32)
    u = np.array([.1, .4, .6, .9], np.float32)
    plain = run(x, u, "plain")
    for kw in (dict(top_p=[NAN] * 4), dict(min_p=[NAN] * 4), dict(top_k=[-5] * 4), dict(top_p=[INF] * 4),
               dict(min_p=[-INF] * 4)):
        ids, probs = run(x, u, kw, **kw)
        assert np.array_equal(ids, plain[0]) and np.array_equal(probs, plain[1])
    ids, probs = run(x, u, "temperature", temperature=[NAN, -1, 0, -INF])
    assert np.array_equal(ids, x.argmax(1)) and (probs == 1).all()


@pytest.mark.parametrize("vocab", [100, 9000, 140000])
def test_rows_of_many_batches(vocab):
    """More rows than one pass of the workspace holds, against calls of a few rows each."""
    m = 1100 if vocab < 100000 else 530
    g = torch.Generator(device=DEV).manual_seed(2)
    x = 4 * torch.randn(m, vocab, device=DEV, generator=g)
    u = torch.rand(m, device=DEV, generator=g)
    t = .5 + torch.rand(m, device=DEV, generator=g)
    k = torch.randint(0, 60, (m,), device=DEV, generator=g).int()
    p = .5 + torch.rand(m, device=DEV, generator=g)
    ids, probs = qlin.sample(qlin.Sampling(t, k, p), x, u)
    for a in range(0, m, 77):
        s = slice(a, min(a + 77, m))
        i, q = qlin.sample(qlin.Sampling(t[s].clone(), k[s].clone(), p[s].clone()), x[s], u[s].clone())
        assert torch.equal(i, ids[s]) and torch.equal(q, probs[s])
    some = [0, 511, 512, m - 1]
    at = torch.tensor(some, device=DEV)
    ref = sr.sample(host(x[at]), host(u[at]), host(t[at]), host(k[at]), host(p[at]))
    sr.check(host(ids)[some], host(probs)[some], ref, vocab)


@pytest.mark.parametrize("vocab", [8192, 8193, 50000, 262144])
def test_flat_rows(vocab):
    """Cuts among more tokens of nearly one logit than are gathered."""
    rng = np.random.default_rng(3)
    x = np.zeros((8, vocab), np.float32)
    x[1:] += (1e-3 * rng.integers(-4, 5, (7, vocab))).astype(np.float32)
    x[4:] += np.where(np.arange(vocab) % 3 == 0, -9.0, 0.0).astype(np.float32)
    u = np.array([.015, .335, .715, .995, .175, .565, .855, .435], np.float32)
    half = vocab // 2

    def check(what, k=None, p=None):
        kw = arrays(top_k=k, top_p=p)
        ids, probs = draw(x, u, *kw)
        rest = []
        for i in range(8):
            order = np.argsort(-x[i], kind="stable")[:vocab if k is None else k[i]]
            if x[i, order[0]] != x[i, order[-1]]:
                rest.append(i)
                continue
            # tokens that weigh the same: sums are whole numbers, exact next to a border too
            n = len(order)
            if p is not None:
                n = math.ceil(Fraction(float(np.float32(p[i]))) * n)
            at = math.floor(Fraction(float(u[i])) * n)
            assert ids[i] == np.sort(order[:n])[at] and probs[i] == np.float32(1 / n), (what, i)
        ref = sr.sample(x[rest], u[rest], *[None if v is None else v[rest] for v in kw])
        sr.check(ids[rest], probs[rest], ref, what)
    k = [half, half, 8000, vocab - 1, half, half + 1, 1000, 9000]
    check("top_k", k=k)
    p = [.3001, .5003, .9007, .0503, .6011, .9907, .9997, .2003]
    check("top_p", p=p)
    check("both", k=[half, half + 3, 8000, vocab - 1, half, vocab - vocab // 6, 1000, 9000], p=p)


def test_cuts_far_apart():
    """top_k far behind top_p, so that two groups of bins are gathered: few and many tokens."""
    rng = np.random.default_rng(4)
    for vocab, k in ((30000, 400), (30000, 20000), (151936, 3000), (151936, 100000)):
        x = (2.5 * rng.standard_normal((6, vocab))).astype(np.float32)
        x[:3, 77] += 12
        run(x, np.array([.02, .51, .98, .11, .66, .87], np.float32), (vocab, k), top_k=[k] * 6,
            top_p=np.array([.31, .52, .9, .43, .7, .95]), min_p=[0, 1e-4, 0, 0, 1e-3, 0])


def test_largest_numbers():
    """Logits of +-the largest number among ordinary ones, at ordinary and tiny temperatures."""
    x = np.zeros((4, 9000), np.float32)
    x[:, 100], x[:, 8500], x[:, 4000], x[:, 4001] = BIG, INF, -BIG, NAN
    run(x, np.array([.2, .4, .6, .9], np.float32), "big", temperature=[1, 1e-38, 3e38, 1],
        top_k=[0, 5, 2, 2])
