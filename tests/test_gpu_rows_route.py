"""GPU parity of qlin_route against the row-by-row 64-bit reference.

ids are equal; a weight is within 2^-20 relative (plus 2^-126): the scores'
exponentials (1 ulp), the softmax's sum over at most 512 terms (tree depth 9),
the division, the renormalization's sum and division and the scale are at most
16 half steps of fp32 together if formed in 32 bits."""
import numpy as np
import pytest
import torch

import rows_ref as rr
from group_wise_bit_amd import qlin

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(logits, top_k, bias=None, **kw):
    r = qlin.Router(logits.shape[1], top_k, bias=None if bias is None else
                    torch.from_numpy(bias).to(DEV), **kw)
    ids, w = qlin.route(r, torch.from_numpy(logits).to(DEV))
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


def check(logits, top_k, label, bias=None, **kw):
    ids, w = run(logits, top_k, bias, **kw)
    rid, rw = rr.route_ref(logits, top_k, bias=bias, **kw)
    assert np.array_equal(ids, rid), f"{label}: ids differ in rows {np.where((ids != rid).any(1))[0][:5]}"
    assert np.all(np.abs(w - rw) <= 2.0 ** -20 * np.abs(rw) + 2.0 ** -126), label


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("m,experts,top_k,groups,top_groups,group_top", [
    (1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (5, 8, 2, 1, 1, 1), (33, 60, 4, 1, 1, 1),
    (7, 63, 8, 1, 1, 2), (64, 64, 8, 8, 4, 2), (9, 65, 5, 5, 2, 1), (130, 128, 8, 4, 1, 1),
    (17, 160, 6, 8, 3, 2), (41, 256, 8, 8, 4, 2), (6, 257, 32, 1, 1, 1), (12, 320, 7, 64, 60, 2),
    (10, 512, 32, 64, 8, 1), (4, 511, 3, 7, 7, 2), (260, 256, 8, 1, 1, 1)])
def test_route(score, with_bias, m, experts, top_k, groups, top_groups, group_top):
    rng = np.random.default_rng([m, experts, top_k])
    logits = (2 * rng.standard_normal((m, experts))).astype(np.float32)
    bias = (0.2 * rng.standard_normal(experts)).astype(np.float32) if with_bias else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        check(logits, top_k, "random", bias, score=score, groups=groups, top_groups=top_groups,
              group_top=group_top, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_ties_masks_and_extremes(score, groups, top_groups):
    inf, low = np.inf, float(np.finfo(np.float32).min)
    rng = np.random.default_rng(3)
    rows = [np.zeros(32), np.full(32, -inf), np.full(32, np.nan), np.full(32, low),
            np.where(np.arange(32) % 3, -inf, 1.5), np.where(np.arange(32) == 17, 2.0, -inf),
            np.where(np.arange(32) < 30, low, 0.0), np.where(np.arange(32) == 5, inf, 0.25),
            np.where(np.arange(32) % 2, inf, -1.0), np.where(np.arange(32) % 4, np.nan, 3.0),
            np.repeat(rng.standard_normal(8), 4), np.full(32, 100.0), np.full(32, -100.0),
            np.linspace(-90, 90, 32), -np.linspace(30, 40, 32),
            np.float32(1.0) + np.arange(32) * np.float32(2.0 ** -23),
            np.float32(0.5) - np.arange(32) * np.float32(2.0 ** -25)]
    logits = np.stack(rows).astype(np.float32)
    for group_top in (1, 2):
        for renorm in (True, False):
            kw = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top,
                      renormalize=renorm)
            if score == "softmax" or group_top == 1:
                check(logits, 6, "no bias", **kw)
            else:
                # (scores that round to one in 64 bits tie there too: left out of the groups' sums)
                check(logits[:14], 6, "no bias", **kw)
            check(logits, 6, "equal bias", np.zeros(32, np.float32), **kw)
            bias = (0.01 * rng.standard_normal(32)).astype(np.float32)
            bias[[3, 9]] = -inf, np.nan
            check(logits, 6, "masking bias", bias, **kw)
            bias[4] = inf
            check(logits, 6, "infinite bias", bias, **kw)
            check(logits, 6, "large bias", (1e6 + np.arange(32)).astype(np.float32), **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_next_to_a_border(score):
    """Biased scores that fp32 cannot tell apart are ordered as in 64 bits."""
    rng = np.random.default_rng(11)
    m, e = 96, 64
    logits = rng.standard_normal((m, e)).astype(np.float32)
    # biases that level the first row's scores to within a few fp32 steps
    x = logits[0].astype(np.float64)
    p = np.exp(x - x.max()) / np.exp(x - x.max()).sum() if score == "softmax" else 1 / (1 + np.exp(-x))
    bias = (0.7 - p).astype(np.float32)
    logits[:] = logits[0]
    logits[np.arange(1, m), rng.integers(0, e, m - 1)] += np.float32(1e-6)
    for kw in (dict(), dict(groups=8, top_groups=3, group_top=2), dict(groups=8, top_groups=3)):
        check(logits, 8, "border", bias, score=score, **kw)


def test_pitch_alignment_and_other_stream():
    rng = np.random.default_rng(5)
    big = torch.from_numpy(rng.standard_normal((37, 131)).astype(np.float32)).to(DEV)
    logits = big[:, 3:123]                    # rows 4-byte aligned only
    r = qlin.Router(120, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ids, w = qlin.route(r, logits)
    side.synchronize()
    rid, rw = rr.route_ref(logits.cpu().numpy(), 5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    ids2, w2 = qlin.route(r, logits.contiguous())
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_empty_batch():
    ids, w = qlin.route(qlin.Router(16, 2), torch.empty(0, 16, device=DEV))
    assert ids.shape == (0, 2) and w.shape == (0, 2)
