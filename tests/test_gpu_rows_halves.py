"""GPU check of how many bits of h = silu(g) * u reach the down product: the fp32 outputs of
qlin_moe_mlp against the 64-bit reference, in every form and at every width.

h is held as two fp16 halves.  The high one is off by 2^-11 |h| at most, the low one, which is
that difference, by 2^-11 of itself: 2^-22 |h| together, or half of fp16's least step, 2^-25.
The rest of the bound counts fp32 roundings as rows_ref.moe_ref does: (k + 8) 2^-24 of the
sum of the terms' sizes for a product over k, 4e-6 for silu (1-ulp exponential and reciprocal,
and the exponential's argument), one rounding each for silu * u and the weight."""
import numpy as np
import pytest
import torch

import rows_forms as rf
import rows_ref as rr
import test_gpu_rows_instances as inst
from test_gpu_rows_moe import call, experts_of, routed

pytestmark = pytest.mark.gpu
U22 = 2.0 ** -22


def reference(x, gate, up, down, ids, wts):
    """(Y, bound of |Y_fp32 - Y|, h of every pair) in binary64."""
    m, top_k = ids.shape
    experts, inner, model = gate.shape
    x = x.astype(np.float64)
    y, err, mag = np.zeros((m, model)), np.zeros((m, model)), np.zeros((m, model))
    hs = np.zeros((m, top_k, inner))
    gk, gi = (model + 8) * rr.U32, (2 * inner + 8) * rr.U32
    for i in range(m):
        for j in range(top_k):
            e = int(ids[i, j])
            if not 0 <= e < experts:
                continue
            ax = np.abs(x[i])
            g, u = gate[e] @ x[i], up[e] @ x[i]
            eg, eu = gk * (np.abs(gate[e]) @ ax), gk * (np.abs(up[e]) @ ax)
            h = rr.silu(g) * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(rr.silu(g)) * eu + (4e-6 + rr.U32) * np.abs(h)
            eh = eh + U22 * (np.abs(h) + eh) + rr.SUB16
            d, ad = down[e] @ h, np.abs(down[e])
            ed = ad @ eh + gi * (ad @ (np.abs(h) + eh))
            w = float(wts[i, j])
            y[i] += w * d
            err[i] += abs(w) * ed
            mag[i] += abs(w) * (np.abs(d) + ed)
            hs[i, j] = h
    return y, err + (top_k + 2) * rr.U32 * mag, hs


def check(ws, what, x, ids, w, label):
    y, y16 = call(ws, x, ids, w)
    ref, err, hs = reference(x, *what, ids, w)
    rr.check(y.cpu().numpy(), ref, err, label)
    rr.check_half(y16.cpu().numpy(), ref, err, label + " fp16")
    return y, ref, hs


# one row (inst.EXPERTS_1); 32 rows with 32 columns, 64, and 64 with K over 4 waves; 64 rows
SIZES = [*inst.EXPERTS_1.values(), (30, 2, 10, 128, 192), (30, 2, 40, 256, 320),
         (40, 3, 120, 192, 192), (660, 1, 16, 1088, 192)]


def rows(rng, m, k):
    return rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)


@pytest.mark.parametrize("bits", inst.WIDTHS)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_bits_of_h(size, bits):
    m, top_k, experts, inner, model = size
    rng = np.random.default_rng([inner, model, bits])
    ws, what = experts_of(rng, experts, inner, model, bits, bits, "64" if bits % 2 else "k")
    ids, w = routed(rng, m, experts, top_k)
    y, ref, _ = check(ws, what, rows(rng, m, model), ids, w, f"{bits} bits")
    # rounding h to one fp16 half leaves 2e-4 here
    assert np.sqrt(np.mean((y.cpu().numpy() - ref) ** 2) / np.mean(ref ** 2)) < 2e-5


@pytest.mark.parametrize("m,experts,inner", [(2, 3, 128), (60, 3, 128), (660, 16, 1088)])
@pytest.mark.parametrize("size", [1e-3, 30.0, 240.0])
def test_small_and_large_h(m, experts, inner, size):
    """h from far below fp16's normal numbers to its largest: rows of x of different sizes."""
    rng = np.random.default_rng([m, int(size)])
    ws, what = experts_of(rng, experts, inner, 256, 4, 4)
    x = (size * rng.standard_normal((m, 256)) * rng.random((m, 1))).astype(np.float16)
    ids, w = routed(rng, m, experts, 1)
    _, _, hs = check(ws, what, x, ids, w, f"size {size}")
    assert np.abs(hs).max() < 65000


@pytest.mark.parametrize("m,experts,inner", [(2, 3, 128), (60, 3, 128), (660, 16, 1088)])
def test_h_beyond_fp16(m, experts, inner):
    """A row with an h from 65520 on is not finite; the others keep every bit."""
    rng = np.random.default_rng(m)
    ws, what = experts_of(rng, experts, inner, 256, 4, 4)
    x = rows(rng, m, 256)
    ids, w = routed(rng, m, experts, 1)
    good, _ = call(ws, x, ids, w)
    x[1] = (x[1].astype(np.float32) * 3000).astype(np.float16)
    _, _, hs = reference(x[1:2], *what, ids[1:2], w[1:2])
    assert np.abs(hs).max() > 70000
    bad, _ = call(ws, x, ids, w)
    keep = np.arange(m) != 1
    assert torch.equal(good[keep], bad[keep])
    assert not torch.isfinite(bad[1]).any()
