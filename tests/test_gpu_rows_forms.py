"""GPU parity of the row-wise products at sizes that take each of their work-group
forms: one row with 8 and 16 columns and 8 and 16 waves, 32 rows with K over 4
and 8 waves, 64 rows with every remainder of its four K stages, many ids to group,
rows further apart than 32-bit offsets reach, ranks above one pass."""
import numpy as np
import pytest
import torch

import rows_ref as rr
from group_wise_bit_amd import qlin
from test_gpu_rows_lora import check as lora_check, dev, pool, weight
from test_gpu_rows_moe import call, check as moe_check, experts_of, routed

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows(rng, m, k):
    return rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)


@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("group", ["64", "k"])
def test_experts_64_rows_every_width(bits, group):
    # 1088 = 17 tiles: the last work-group's second half is past the matrix
    rng = np.random.default_rng([1, bits, len(group)])
    ws, what = experts_of(rng, 16, 1088, 192, bits, 10 - bits, group)
    ids, w = routed(rng, 660, 16, 1)
    ids[rng.random(ids.shape) < 0.05] = -1
    moe_check(ws, what, rows(rng, 660, 192), ids, w, f"{bits} bits")


@pytest.mark.parametrize("model", [64, 128, 256, 320, 448])
def test_experts_64_rows_k_remainders(model):
    rng = np.random.default_rng(model)
    ws, what = experts_of(rng, 8, 1024, model, 4, 3)
    x = rows(rng, 700, model)
    ids, w = routed(rng, 700, 8, 2)
    moe_check(ws, what, x, ids, w, "spread")
    ids[:] = np.where(ids < 4, 6, -1)            # one expert, half of the slots
    moe_check(ws, what, x, ids, w, "one expert")


@pytest.mark.parametrize("inner,model", [(128, 2112), (2112, 128), (576, 576)])
@pytest.mark.parametrize("bits,dbits", [(3, 6), (8, 3), (6, 4)])
def test_experts_32_rows_k_over_waves(inner, model, bits, dbits):
    rng = np.random.default_rng([inner, model, bits])
    ws, what = experts_of(rng, 64, inner, model, bits, dbits)
    moe_check(ws, what, rows(rng, 40, model), *routed(rng, 40, 64, 2), "64 experts")


@pytest.mark.parametrize("m,experts,top_k,inner,model,bits", [
    (1, 8, 8, 512, 2112, 4),      # gate and up: 16 columns, 16 waves
    (1, 40, 32, 64, 4096, 4),     # more slots than waves, 16 columns
    (1, 20, 20, 64, 64, 7),       # 8 waves for 20 slots, 8 columns
    (2, 16, 16, 192, 256, 2),     # as many slots as waves
    (4, 3, 3, 320, 4096, 5),
    (32, 2, 1, 64, 128, 8)])      # the most pairs that go alone
def test_experts_one_row_forms(m, experts, top_k, inner, model, bits):
    rng = np.random.default_rng([m, experts, inner])
    ws, what = experts_of(rng, experts, inner, model, bits, bits)
    x = rows(rng, m, model)
    ids, w = routed(rng, m, experts, top_k)
    moe_check(ws, what, x, ids, w, "random")
    moe_check(ws, what, x, np.full_like(ids, 1), w, "the same expert in every slot")
    ids[:, ::2] = -1
    moe_check(ws, what, x, ids, w, "every other slot empty")


def test_experts_too_large_to_go_alone():
    rng = np.random.default_rng(3)
    ws, what = experts_of(rng, 2, 1792, 4096, 8, 8)
    for m in (2, 3):                             # 88 MB alone; 132 MB grouped
        moe_check(ws, what, rows(rng, m, 4096), *routed(rng, m, 2, 2), f"m={m}")


@pytest.mark.parametrize("m,experts,top_k", [(5000, 3, 2), (8300, 1, 1), (4200, 512, 2)])
def test_many_ids_to_group(m, experts, top_k):
    rng = np.random.default_rng(m)
    ws, what = experts_of(rng, experts, 64, 64, 4, 4)
    ids, w = routed(rng, m, experts, top_k)
    ids[rng.random(ids.shape) < 0.1] = experts
    moe_check(ws, what, rows(rng, m, 64), ids, w, "many ids")


@pytest.mark.parametrize("m", [8191, 8193, 66000, 540000])
def test_many_ids_of_few_kinds(m):
    """Rows of 5 kinds through 3 experts or none: 20 results, each at its rows."""
    rng = np.random.default_rng(m)
    ws, what = experts_of(rng, 3, 64, 64, 4, 4)
    kinds = rows(rng, 5, 64)
    kind, e = rng.integers(0, 5, m), rng.integers(-1, 3, m)
    ref, err = rr.moe_ref(np.repeat(kinds, 4, 0), *what, np.tile(np.arange(-1, 3, dtype=np.int32), 5)[:, None],
                          np.ones((20, 1), np.float32))
    y, _ = call(ws, kinds[kind], e.astype(np.int32)[:, None], np.ones((m, 1), np.float32))
    at = 4 * kind + e + 1
    rr.check(y.cpu().numpy(), ref[at], err[at], f"{m} ids")


def test_rows_far_apart():
    """Rows of X over more than 4 GB take the forms with 64-bit addresses."""
    m, pitch = 660, 1 << 22
    store = torch.zeros(m * pitch, dtype=torch.float16, device=DEV)
    rng = np.random.default_rng(5)
    ws, what = experts_of(rng, 16, 1088, 128, 4, 4)
    x = rows(rng, m, 128)
    X = store.view(m, pitch)[:, :128]
    X.copy_(dev(x))
    ids, w = routed(rng, m, 16, 1)
    y, _ = qlin.moe_mlp(*ws, X, dev(ids), dev(w))
    rr.check(y.cpu().numpy(), *rr.moe_ref(x, *what, ids, w), "experts")
    p = pool(rng, 3, 4096, 128, 16)
    wq, wh = weight(rng, 4096, 128, 4, 64)
    aid = rng.integers(-1, 3, m).astype(np.int32)
    y, _ = qlin.gemm_lora(wq, X, qlin.Adapters(*map(dev, p)), dev(aid))
    rr.check(y.cpu().numpy(), *rr.lora_ref(x, wh, *p, aid), "adapters")


@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("group", ["64", "k"])
def test_adapters_64_rows_every_width(bits, group):
    rng = np.random.default_rng([2, bits, len(group)])
    n, k, m = 9200, 64 * (1 + bits % 5), 250
    w, what = weight(rng, n, k, bits, 64 if group == "64" else k)
    ids = rng.integers(-1, 3, m).astype(np.int32)
    lora_check(w, what, rows(rng, m, k), pool(rng, 3, n, k, 16), ids, f"{bits} bits")


@pytest.mark.parametrize("rank", [8, 24, 64, 72, 128])
@pytest.mark.parametrize("order", ["sorted", "mixed", "none", "one"])
def test_adapters_64_rows_ranks(rank, order):
    rng = np.random.default_rng([rank, len(order)])
    n, k, m, slots = 4160, 576, 580, 9
    w, what = weight(rng, n, k, 4, 64)
    ids = rng.integers(-2, slots + 1, m).astype(np.int32)
    if order == "sorted":
        ids.sort()
    elif order == "none":
        ids[:] = -1
    elif order == "one":
        ids[:] = 7
    lora_check(w, what, rows(rng, m, k), pool(rng, slots, n, k, rank, rank != 24), ids, order)


@pytest.mark.parametrize("m,n,k", [(20, 8192, 128), (20, 8192, 576), (20, 8192, 2112),
                                   (40, 4128, 1024), (33, 64, 2112)])
@pytest.mark.parametrize("rank", [8, 128])
def test_adapters_32_rows_k_over_waves(m, n, k, rank):
    rng = np.random.default_rng([m, n, k, rank])
    w, what = weight(rng, n, k, 4, 64)
    ids = rng.integers(-1, 40, m).astype(np.int32)
    lora_check(w, what, rows(rng, m, k), pool(rng, 40, n, k, rank), ids, "mixed")


@pytest.mark.parametrize("m", [160, 700])
def test_adapters_ordered_32_rows(m):
    rng = np.random.default_rng(m)
    w, what = weight(rng, 200, 448, 5, 64)
    ids = rng.integers(-1, 6, m).astype(np.int32)
    lora_check(w, what, rows(rng, m, 448), pool(rng, 6, 200, 448, 128), ids, "ordered")


def test_workspace_grows_between_calls_and_graphs():
    """Small, large, small again on one stream, a graph between them: each call's result
    is its own, and the graph's does not change when the cached workspace grows."""
    rng = np.random.default_rng(9)
    ws, _ = experts_of(rng, 8, 1024, 256, 4, 4)
    sizes = (1, 40, 700)
    args = {m: [dev(t) for t in (rows(rng, m, 256), *routed(rng, m, 8, 2))] for m in sizes}
    first = {m: qlin.moe_mlp(*ws, *args[m])[0].clone() for m in sizes}
    qlin._WS.clear()
    assert torch.equal(qlin.moe_mlp(*ws, *args[1])[0], first[1])
    graphs = {}
    for m in (40, 700):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = qlin.moe_mlp(*ws, *args[m])[0]
        graphs[m] = g, out
    big = qlin.moe_mlp(*ws, *args[700])[0]
    for _ in range(3):
        for m in (40, 700):
            graphs[m][0].replay()
        small = qlin.moe_mlp(*ws, *args[1])[0]
        torch.cuda.synchronize()
        assert all(torch.equal(graphs[m][1], first[m]) for m in graphs)
        assert torch.equal(small, first[1]) and torch.equal(big, first[700])


@pytest.mark.parametrize("m", [40, 700])
def test_experts_64_rows_do_not_mix(m):
    """Rows that are not finite stay alone, on 64-row tiles as well."""
    rng = np.random.default_rng(m)
    ws, _ = experts_of(rng, 8, 1024, 256, 4, 4)
    x = rows(rng, m, 256)
    ids, w = routed(rng, m, 8, 2)
    good, _ = call(ws, x, ids, w)
    x[7, 3], x[31, 255] = np.nan, np.inf
    bad, _ = call(ws, x, ids, w)
    keep = np.setdiff1d(np.arange(m), [7, 31])
    assert torch.equal(good[keep], bad[keep])
    assert not torch.isfinite(bad[7]).any() and not torch.isfinite(bad[31]).any()
