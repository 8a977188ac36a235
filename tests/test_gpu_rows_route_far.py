"""GPU parity of qlin_route where 32 bits are furthest from enough: the chosen experts far
below the row's largest logit (which a bias masks or outranks).  Reference and tolerance are
those of test_gpu_rows_route.py: equal ids, weights within 2^-20 relative plus 2^-126."""
import numpy as np
import pytest

from test_gpu_rows_route import check

pytestmark = pytest.mark.gpu

GAPS = (60, 79, 81, 85, 88, 95, 100, 103, 105, 150, 300, 700)


def below(rng, gap, experts, tops):
    """Rows whose best logit (at each of tops in turn) stands gap above the others' best."""
    x = (-3 * rng.random((len(tops), experts))).astype(np.float32)
    x[:, 1::7] = 0
    x[np.arange(len(tops)), tops] = gap
    return x


@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("top_k", [1, 2, 6])
@pytest.mark.parametrize("mask", ["inf", "nan", "outranked"])
def test_chosen_far_below_the_largest(mask, top_k, groups, top_groups, group_top):
    rng = np.random.default_rng([top_k, groups, group_top])
    bias = (0.1 + 0.05 * rng.permutation(24)).astype(np.float32)
    bias[5] = {"inf": -np.inf, "nan": np.nan, "outranked": -9.0}[mask]
    for gap in GAPS:
        logits = below(rng, gap, 24, [5] * 9)
        for renorm, scale in ((True, 1.5), (False, 1.0), (False, 1e25)):
            check(logits, top_k, f"gap {gap}", bias, score="softmax", groups=groups,
                  top_groups=top_groups, group_top=group_top, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("gap", GAPS)
def test_some_chosen_far_below(gap):
    """One or two near the top, the others far below it; and a gap inside the chosen alone."""
    rng = np.random.default_rng(gap)
    logits = below(rng, gap, 40, np.arange(40) % 13)
    logits[::2, 20] = gap - 1.0
    check(logits, 5, "near and far", score="softmax")
    check(logits, 5, "near and far", (0.01 * np.arange(40)).astype(np.float32), score="softmax")
    bias = np.full(40, 4.0, np.float32)
    bias[:13] = -np.inf
    logits[:, 30] = gap - 59.0
    check(logits, 5, "far, with a gap of its own", bias, score="softmax")
