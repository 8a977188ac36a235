"""GPU parity of qlin_route where groups of experts are hard to tell apart in 32 bits: two
best biased scores that are large and of opposite sign, sums beyond fp32's range, masks made
of large negative biases.  Reference and tolerance are those of test_gpu_rows_route.py."""
import numpy as np
import pytest

from test_gpu_rows_route import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1.0, 64.0, 1000.0, 65536.0, 1e6])
def test_groups_of_opposite_biases(score, size):
    """The sum of a group's two best is small, each of them is rounded at its own size."""
    rng = np.random.default_rng(int(size))
    groups, per, m = 8, 4, 200
    bias = np.tile(np.array([size, -size, -4 * size, -3 * size], np.float32), groups)
    one = rng.standard_normal((m, 1, per))
    near = np.broadcast_to(one, (m, groups, per)) + 1e-6 * rng.standard_normal((m, groups, per))
    apart = rng.standard_normal((m, groups, per))
    for x in (near, apart):
        logits = np.clip(x, -3, 3).reshape(m, -1).astype(np.float32)
        for top_groups in (1, 3, 7):
            check(logits, 4, f"top {top_groups}", bias, score=score, groups=groups,
                  top_groups=top_groups, group_top=2)
    # a group whose second best is masked by a large negative bias does not blur the others
    wide = rng.permuted(np.tile(np.array([0.3, 0.2, -size, -1e9], np.float32), (groups, 1)), axis=1)
    check(rng.standard_normal((m, groups * per)).astype(np.float32), 4, "masked by size",
          wide.reshape(-1), score=score, groups=groups, top_groups=3, group_top=2)
    lone = np.tile(np.array([0.3, -1e9, -1e9, -1e9], np.float32), groups)
    check(rng.standard_normal((m, groups * per)).astype(np.float32), 3, "one of a group",
          lone, score=score, groups=groups, top_groups=3, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_values_beyond_32_bits(score):
    """Biases whose sums exceed fp32's range are still ordered."""
    rng = np.random.default_rng(7)
    big = 3e38
    bias = np.array([big, big, 0, 0, big, 2e38, 0, 0, -big, -big, -big, -big, 1, 1, 1, 1], np.float32)
    logits = rng.standard_normal((20, 16)).astype(np.float32)
    for top_groups in (1, 2, 3, 4):
        check(logits, 4, f"top {top_groups}", bias, score=score, groups=4, top_groups=top_groups,
              group_top=2)
