"""GPU parity of qlin_gemm_lora against the 64-bit reference, within the derived
bounds of rows_ref: every width, row counts from one to several tiles, ranks,
rows with and without adapters in any order, pitches, streams, capture; and
routing, experts and adapters run one after the other as a layer does."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import rows_ref as rr
from group_wise_bit_amd import qlin

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weight(rng, n, k, bits, group):
    w, s, z, what = rr.packed_stack(rng, 1, n, k, bits, group)
    return qlin.QWeight(n, k, bits, group, qlin.FMT_PACKED, torch.from_numpy(w).to(DEV),
                        torch.from_numpy(s).to(DEV), torch.from_numpy(z).to(DEV)), what[0]


def pool(rng, slots, n, k, rank, scaled=True):
    a = (rng.standard_normal((slots, rank, k)) / np.sqrt(k)).astype(np.float16)
    b = (0.3 * rng.standard_normal((slots, n, rank))).astype(np.float16)
    s = (rng.random(slots) * 3 - 1).astype(np.float32) if scaled else None
    return a, b, s


def dev(t):
    return None if t is None else torch.from_numpy(np.ascontiguousarray(t)).to(DEV)


def check(w, what, x, abs_, ids, label):
    a, b, s = abs_
    y, y16 = qlin.gemm_lora(w, dev(x), qlin.Adapters(dev(a), dev(b), dev(s)), dev(ids))
    torch.cuda.synchronize()
    ref, err = rr.lora_ref(x, what, a, b, s, ids)
    rr.check(y.cpu().numpy(), ref, err, label)
    rr.check_half(y16.cpu().numpy(), ref, err, label + " fp16")
    assert torch.equal(y.half(), y16), label
    return y


@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("group", [64, "k"])
def test_every_width(bits, group):
    rng = np.random.default_rng([bits, 1 if group == 64 else 2])
    n, k = 200, 320
    w, what = weight(rng, n, k, bits, 64 if group == 64 else k)
    p = pool(rng, 4, n, k, 16)
    for m in (1, 19, 150, 300):
        x = rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)
        check(w, what, x, p, rng.integers(-1, 4, m).astype(np.int32), f"{bits} bits m={m}")


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 64, 65, 128, 129, 257, 400])
@pytest.mark.parametrize("n,k,rank,slots", [(1, 64, 8, 1), (63, 128, 24, 3), (65, 64, 40, 70),
                                            (192, 448, 64, 2), (130, 1024, 128, 5)])
def test_sizes(m, n, k, rank, slots):
    rng = np.random.default_rng([m, n, rank])
    w, what = weight(rng, n, k, 4, 64)
    p = pool(rng, slots, n, k, rank, scaled=m % 2 == 0)
    x = rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)
    check(w, what, x, p, rng.integers(-1, slots, m).astype(np.int32), "mixed")
    check(w, what, x, p, np.sort(rng.integers(0, slots, m)).astype(np.int32), "sorted")
    check(w, what, x, p, np.full(m, slots - 1, np.int32), "one adapter")


@pytest.mark.parametrize("m", [5, 200, 300])
def test_rows_without_adapters(m):
    rng = np.random.default_rng(m)
    n, k = 96, 256
    w, what = weight(rng, n, k, 4, 64)
    p = pool(rng, 3, n, k, 16)
    x = rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)
    none = np.full(m, -1, np.int32)
    none[0], none[-1] = 3, 2 ** 31 - 1
    y = check(w, what, x, p, none, "no adapters")
    # a NaN adapter that no row asks for is not seen
    p[0][1], p[1][1], p[2][1] = np.nan, np.nan, np.nan
    ids = rng.choice([-1, 0, 2], m).astype(np.int32)
    check(w, what, x, p, ids, "an unused adapter of NaN")
    # rows whose adapter is not finite are their own affair
    y0, _ = qlin.gemm_lora(w, dev(x), qlin.Adapters(*map(dev, p)), dev(none))
    mixed = none.copy()
    mixed[1] = 1
    y1, _ = qlin.gemm_lora(w, dev(x), qlin.Adapters(*map(dev, p)), dev(mixed))
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(y0, y) and torch.equal(y0[keep], y1[keep]) and torch.isnan(y1[1]).all()
    p[0][1], p[1][1], p[2][1] = 0, np.inf, 1
    y2, _ = qlin.gemm_lora(w, dev(x), qlin.Adapters(*map(dev, p)), dev(mixed))
    assert torch.equal(y0[keep], y2[keep])


@pytest.mark.parametrize("m", [4, 300])
def test_ranges_of_the_first_product(m):
    """A x of any finite size keeps its 22 bits: far above fp16's end and far below its start."""
    rng = np.random.default_rng(m)
    n, k = 64, 128
    w, what = weight(rng, n, k, 4, 64)
    a, b, _ = pool(rng, 4, n, k, 8)
    a[0] *= 4096
    a[1] = (a[1].astype(np.float64) * 1e-3).astype(np.float16)
    s = np.array([3e4, 1e-9, 0.0, -1e30], np.float32)
    x = (100 * rng.standard_normal((m, k))).astype(np.float16)
    check(w, what, x, (a, b, s), (np.arange(m) % 5 - 1).astype(np.int32), "ranges")


@pytest.mark.parametrize("m", [7, 290])
def test_pitches_outputs_and_workspaces(m):
    rng = np.random.default_rng(m)
    n, k = 150, 192
    w, what = weight(rng, n, k, 6, 64)
    p = pool(rng, 3, n, k, 8)
    ad = qlin.Adapters(*map(dev, p))
    x = rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)
    ids = dev(rng.integers(-1, 3, m).astype(np.int32))
    y, y16 = qlin.gemm_lora(w, dev(x), ad, ids)
    X = torch.zeros(m, 256, dtype=torch.float16, device=DEV)
    X[:, 8:200] = dev(x)
    Y = torch.full((m + 1, 155), 7.0, device=DEV)
    Y16 = Y.half()
    qlin.gemm_lora(w, X[:, 8:200], ad, ids, Y=Y, Y16=Y16)
    assert torch.equal(Y[:m, :n], y) and torch.equal(Y16[:m, :n], y16)
    assert (Y[m:] == 7).all() and (Y[:, n:] == 7).all() and (Y16[:, n:] == 7).all()
    assert torch.equal(qlin.gemm_lora(w, X[:, 8:200], ad, ids, want_y16=False)[0], y)
    assert torch.equal(qlin.gemm_lora(w, X[:, 8:200], ad, ids, want_y=False)[1], y16)
    need = qlin.library().qlin_gemm_lora_workspace_bytes(
        ctypes.byref(w.c_struct()), ctypes.byref(ad.c_struct(w)), m)
    for fill in (0, 255, 127):
        mine = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        y2, _ = qlin.gemm_lora(w, dev(x), ad, ids, ws=mine[:need])
        assert torch.equal(y2, y)
        assert (mine[:65536] == fill).all() and (mine[need:] == fill).all()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_reruns_streams_and_capture(m):
    rng = np.random.default_rng(m)
    n, k = 130, 512
    w, _ = weight(rng, n, k, 4, 64)
    ad = qlin.Adapters(*map(dev, pool(rng, 6, n, k, 16)))
    mk = lambda: (dev(rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)),  # noqa: E731
                  dev(rng.integers(-1, 6, m).astype(np.int32)))
    x, ids = mk()
    y, _ = qlin.gemm_lora(w, x, ad, ids)
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            outs += [qlin.gemm_lora(w, x, ad, ids)[0] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gy16 = qlin.gemm_lora(w, x, ad, ids)
    for _ in range(4):
        nx, nids = mk()
        x.copy_(nx), ids.copy_(nids)
        graph.replay()
        eager, eager16 = qlin.gemm_lora(w, x.clone(), ad, ids.clone())
        torch.cuda.synchronize()
        assert torch.equal(gy, eager) and torch.equal(gy16, eager16)


def test_agrees_with_the_dense_call():
    """Without adapters the product is qlin_gemm's, to the matmul contract."""
    rng = np.random.default_rng(4)
    for n, k, m in ((896, 896, 8), (320, 4864, 1), (512, 1024, 300)):
        w, what = weight(rng, n, k, 4, 64)
        x = rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)
        ad = qlin.Adapters(*map(dev, pool(rng, 1, n, k, 8)))
        y, _ = qlin.gemm_lora(w, dev(x), ad, dev(np.full(m, -1, np.int32)))
        off = float((y - qlin.gemm(w, dev(x))).abs().max())
        assert off <= 1e-3 * oracle.tolerance_scale(x, what)


@pytest.mark.parametrize("m", [1, 24, 300])
def test_a_layer_of_them(m):
    """Projection with adapters -> router -> experts, and adapters on the way out, one
    after the other on one stream, captured as a whole and replayed."""
    rng = np.random.default_rng(m)
    model, inner, experts, top_k = 256, 128, 8, 2
    proj, wproj = weight(rng, model, model, 4, 64)
    p = pool(rng, 3, model, model, 8)
    ad = qlin.Adapters(*map(dev, p))
    wr = dev((rng.standard_normal((experts, model)) / 16).astype(np.float32))
    gate, wg = (lambda t: (qlin.QExperts(experts, inner, model, 4, 64, dev(t[0]), dev(t[1]), dev(t[2])),
                           t[3]))(rr.packed_stack(rng, experts, inner, model, 4, 64))
    up, wu = (lambda t: (qlin.QExperts(experts, inner, model, 4, 64, dev(t[0]), dev(t[1]), dev(t[2])),
                         t[3]))(rr.packed_stack(rng, experts, inner, model, 4, 64))
    down, wd = (lambda t: (qlin.QExperts(experts, model, inner, 3, 64, dev(t[0]), dev(t[1]), dev(t[2])),
                           t[3]))(rr.packed_stack(rng, experts, model, inner, 3, 64))
    router = qlin.Router(experts, top_k, score="sigmoid", bias=dev(np.linspace(0, .1, experts, dtype=np.float32)),
                         groups=4, top_groups=2)
    x = dev(rng.standard_normal((m, model), dtype=np.float32).astype(np.float16))
    lid = dev(rng.integers(-1, 3, m).astype(np.int32))

    def layer():
        y, h = qlin.gemm_lora(proj, x, ad, lid)
        logits = h.float() @ wr.t()
        ids, w = qlin.route(router, logits)
        o, o16 = qlin.moe_mlp(gate, up, down, h, ids, w)
        z, _ = qlin.gemm_lora(proj, o16, ad, lid, want_y16=False)
        return h, logits, ids, w, o, o16, z
    h, logits, ids, w, o, o16, z = layer()
    torch.cuda.synchronize()
    host = lambda t: t.cpu().numpy()  # noqa: E731
    ref, err = rr.lora_ref(host(x), wproj, *p, host(lid))
    rr.check_half(host(h), ref, err, "projection")
    rid, rw = rr.route_ref(host(logits), top_k, score="sigmoid", bias=host(router.bias), groups=4,
                           top_groups=2)
    assert np.array_equal(host(ids), rid)
    ref, err = rr.moe_ref(host(h), wg, wu, wd, rid, host(w))
    rr.check(host(o), ref, err, "experts")
    ref, err = rr.lora_ref(host(o16), wproj, *p, host(lid))
    rr.check(host(z), ref, err, "out projection")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        graph.replay()
        eager = layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
