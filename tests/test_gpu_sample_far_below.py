"""Drawing tokens of which thousands lie far below another, over several slices of the row: their
sums are as fine as the header says."""
import numpy as np
import pytest

from test_gpu_sample import arrays, draw

pytestmark = pytest.mark.gpu


def check(x, u, ids, probs, k, p):
    """The drawn token's place among the sums of exact arithmetic, within twice the header's
    2^-34 + vocab * 2^-45 (a border of top_p's and the one of u)."""
    vocab = x.shape[1]
    tol = 2 * (2.0 ** -34 + vocab * 2.0 ** -45)
    for i in range(len(u)):
        row = x[i].astype(np.float64)
        order = np.argsort(-row, kind="stable")[:k[i]]
        mass = np.exp(row[order] - row.max())
        if p is not None:
            n = 1 + int((np.cumsum(mass) < float(np.float32(p[i])) * mass.sum()).sum())
            order, mass = order[:n], mass[:n]
        by = np.argsort(order)
        order, mass = order[by], mass[by]
        sums = np.cumsum(mass) / mass.sum()
        where = np.flatnonzero(order == ids[i])
        # (a token next to top_p's border may be kept or not)
        at = int(where[0]) if len(where) else int(np.searchsorted(order, ids[i]))
        target = float(u[i])
        assert sums[max(at - 1, 0)] * (at > 0) <= target + tol, (i, ids[i], at)
        assert sums[min(at, len(sums) - 1)] >= target - tol, (i, ids[i], at)
        w = np.exp(row[ids[i]] - row.max()) / mass.sum()
        assert abs(probs[i] - w) <= (2.0 ** -23 + tol) * w, (i, probs[i], w)


@pytest.mark.parametrize("depth", [120, 200, 290])
@pytest.mark.parametrize("vocab,ties", [(30000, 7000), (151936, 8000), (60000, 600)])
def test_many_far_below(depth, vocab, ties):
    """One token, and equal ones `depth` twelfths below its logit, the cut of top_k among them and
    that of top_p anywhere from the first token on: every sum is over all of them."""
    rng = np.random.default_rng(depth + vocab)
    m = 24
    x = np.full((m, vocab), -80, np.float32)
    top = vocab - 1 - np.arange(m) * (vocab // m // 2)
    for i in range(m):
        at = rng.permutation(vocab - 1)[:ties]
        x[i, at] = -depth / 12
        x[i, top[i]] = 0.0
    one = np.exp(-depth / 12)
    # from 0 on to the sum of those before the one token, and behind it
    u = np.empty(m, np.float32)
    u[:12] = rng.random(12) * 0.4 * ties * one / (1 + ties * one)
    u[12:] = 1 - np.arange(1, 13) * 2.0 ** -24
    k = np.full(m, ties - 10, np.int32)
    p = np.full(m, np.float32(1) - np.float32(2.0 ** -24))
    kw = arrays(top_k=k, top_p=p)
    ids, probs = draw(x, u, *kw)
    check(x, u, ids, probs, k, p)
    ids, probs = draw(x, u, *arrays(top_k=k))
    check(x, u, ids, probs, k, None)
