"""Drawing tokens where logits of +0 and -0 stand side by side: they are equal, and go by index."""
import numpy as np
import pytest

from test_gpu_sample import arrays, draw

pytestmark = pytest.mark.gpu
LAST = float(np.nextafter(np.float32(1), np.float32(0)))


def test_few_tokens():
    x = np.array([[-0.0, 0.0, 0.0], [0.0, -0.0, 0.0], [-0.0, -0.0, 0.0], [-1.0, -0.0, 0.0]], np.float32)
    u = np.full(4, LAST, np.float32)
    ids, _ = draw(x, u, *arrays(top_k=[2] * 4))
    assert ids.tolist() == [1, 1, 1, 2]
    ids, _ = draw(x, u, *arrays(top_p=[0.6, 0.6, 0.6, 0.3]))
    assert ids.tolist() == [1, 1, 1, 1]
    ids, _ = draw(x, u * 0, *arrays(top_k=[2] * 4))
    assert ids.tolist() == [0, 0, 0, 1]
    for kw in (dict(top_k=[1] * 4), dict(temperature=[0] * 4), dict(top_p=[0] * 4), dict(min_p=[2] * 4)):
        ids, probs = draw(x, u, *arrays(**kw))
        assert ids.tolist() == [0, 0, 0, 1] and (probs == 1).all(), kw


@pytest.mark.parametrize("vocab,zeros", [(600, 400), (20000, 3000), (40000, 20000)])
def test_cuts_among_zeros(vocab, zeros):
    """Zeros of both signs among far lower tokens: in the list of few tokens, in that of many, and
    more than are listed."""
    rng = np.random.default_rng(1)
    x = np.full((6, vocab), -60, np.float32)
    at = np.stack([np.sort(rng.permutation(vocab)[:zeros]) for _ in range(6)])
    for i in range(6):
        x[i, at[i]] = np.where(rng.random(zeros) < 0.5, np.float32(-0.0), np.float32(0.0))
    x[3:, 7] = 1.0                               # a token above them
    k = np.array([zeros // 2, zeros // 3, 2, zeros // 2, zeros // 5, 10], np.int32)
    zeros_kept = k - (np.arange(6) >= 3)

    def last_and_first(kept_zeros, *settings):
        want = []
        for i in range(6):
            kept = np.union1d([] if i < 3 else [7], [j for j in at[i] if j != 7 or i < 3][:kept_zeros[i]])
            want.append((int(kept[0]), int(kept[-1])))
        for u, side in ((0.0, 0), (LAST, 1)):
            ids, _ = draw(x, np.full(6, u, np.float32), *settings)
            assert ids.tolist() == [w[side] for w in want]
    last_and_first(zeros_kept, *arrays(top_k=k))
    # half of the zeros' mass, in the middle of a token
    e = np.exp(1.0) * (np.arange(6) >= 3)
    half = zeros // 2
    n = np.array([zeros if 7 not in at[i] or i < 3 else zeros - 1 for i in range(6)])
    last_and_first(np.full(6, half), *arrays(top_p=(half - 0.5 + e) / (n + e)))
