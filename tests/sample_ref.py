"""64-bit reference of drawing a token (include/qlin_sample.h), from its definition.  It also says
how close a row's choice is to a border: `margin`, relative to the sums that are compared."""
import numpy as np


def kept_tokens(row, t, k, p, mp):
    """(indices of the kept tokens in the order, p of each, distance of the cut from another)."""
    x = np.minimum(np.where(np.isnan(row), -np.inf, row.astype(np.float64)), np.finfo(np.float32).max)
    here = np.flatnonzero(x > -np.inf)
    order = here[np.argsort(-x[here], kind="stable")]
    if not len(order):
        return order, np.zeros(0), 1.0
    if not t > 0 or k == 1:
        return order[:1], np.ones(1), 1.0
    mass = np.exp((x[order] - x[order[0]]) / float(np.float32(t)))
    margin = 1.0
    if k > 0:
        order, mass = order[:k], mass[:k]
    n = len(order)
    if p < 1:
        target = max(float(np.float32(p)), 0.0) * mass.sum()
        sums = np.cumsum(mass)
        n = 1 + int((sums < target).sum())
        n = min(n, len(order))
        near = np.abs(sums - target) / mass.sum()
        if target > 0:
            margin = min(margin, near[max(n - 2, 0):n + 1].min())
    if mp > 0:
        limit = float(np.float32(mp))
        n = min(n, max(1, int((mass >= limit).sum())))
        if len(mass) > 1:
            margin = min(margin, np.abs(mass[1:] / limit - 1).min())
    return order[:n], mass[:n], margin


def sample_row(row, u, t=1.0, k=0, p=1.0, mp=0.0):
    """(id, probability, margin)."""
    order, mass, margin = kept_tokens(row, t, k, p, mp)
    if not len(order):
        return -1, 0.0, 1.0
    by_index = np.argsort(order)
    order, mass = order[by_index], mass[by_index]
    sums = np.cumsum(mass)
    target = (float(np.float32(u)) if u > 0 else 0.0) * sums[-1]
    at = int((sums <= target).sum())
    margin = min(margin, np.abs(sums[max(at - 1, 0):at + 1] - target).min() / sums[-1]
                 if 0 < target < sums[-1] else 1.0)
    if at >= len(order):
        at = int(np.flatnonzero(mass > 1e-16)[-1])
    return int(order[at]), mass[at] / sums[-1], margin


def setting(v, i, off):
    return off if v is None else v[i]


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    rows = [sample_row(logits[i], u[i], setting(temperature, i, 1.0), setting(top_k, i, 0),
                       setting(top_p, i, 1.0), setting(min_p, i, 0.0)) for i in range(len(u))]
    return tuple(np.array(x) for x in zip(*rows))


def check(ids, probs, ref, what):
    """Equal ids -- but where a border is within 2^-28 of the choice, which no drawn row should be
    -- and probabilities to 2^-23 (one rounding to fp32, and one of the test's sums)."""
    want, wp, margin = ref
    sure = margin > 2.0 ** -28
    assert sure.all(), (what, "a row next to a border", margin.min())
    assert np.array_equal(ids, want), (what, np.flatnonzero(ids != want)[:5], ids[ids != want][:5],
                                       want[ids != want][:5])
    assert np.all(np.abs(probs - wp) <= 2.0 ** -23 * wp), what
