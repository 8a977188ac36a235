"""GPU parity of every work-group instance of the row-wise products at every width: the
one-row form with 8 and 16 columns and 8 and 16 waves; the 32-row form with 32 columns, with
64 and K over 8 waves, with 64 and K over 4, for experts and for adapters added by threads,
on the matrix cores, and over rows ordered by adapter.  tests/test_rows_form_sizes.py holds
each size here to the form it is named for."""
import numpy as np
import pytest

from test_gpu_rows_lora import check as lora_check, pool, weight
from test_gpu_rows_moe import check as moe_check, experts_of, routed

pytestmark = pytest.mark.gpu
WIDTHS = (2, 3, 4, 5, 6, 7, 8)

# m, n, rank of adapters by (how they are added, columns, waves)
ADAPTERS = {
    ("dots", 32, 8): (96, 200, 24), ("dots", 64, 8): (96, 4150, 8), ("dots", 64, 4): (96, 8190, 32),
    ("come", 32, 8): (90, 200, 40), ("come", 64, 8): (90, 4150, 128), ("come", 64, 4): (90, 8190, 64),
    ("ordered", 32, 8): (161, 200, 128), ("ordered", 64, 8): (161, 2000, 128),
    ("ordered", 64, 4): (161, 4150, 128),
}
# low ranks of ordered rows
ORDERED = [(700, 200, 32), (700, 640, 48), (700, 1088, 32), (1300, 960, 16)]

# m, top_k, experts, inner, model of experts by (columns, waves), of both products
EXPERTS_32 = {(32, 8): (30, 2, 40, 128, 192), (64, 8): (30, 2, 40, 256, 320),
              (64, 4): (30, 2, 40, 512, 576)}
EXPERTS_1 = {(16, 8): (8, 2, 5, 256, 512), (8, 8): (3, 2, 4, 128, 192),
             (8, 16): (1, 2, 3, 1088, 2112)}


def rows(rng, m, k):
    return rng.standard_normal((m, k), dtype=np.float32).astype(np.float16)


@pytest.mark.parametrize("bits", WIDTHS)
@pytest.mark.parametrize("form", ADAPTERS, ids=lambda f: "-".join(map(str, f)))
def test_adapters(form, bits):
    m, n, rank = ADAPTERS[form]
    rng = np.random.default_rng([m, n, rank, bits])
    k = 64 * (2 + bits % 4)
    w, what = weight(rng, n, k, bits, 64 if bits % 2 else k)
    ids = rng.integers(-1, 6, m).astype(np.int32)
    lora_check(w, what, rows(rng, m, k), pool(rng, 6, n, k, rank), ids, "mixed")


@pytest.mark.parametrize("m,n,rank", ORDERED)
def test_adapters_ordered_low_ranks(m, n, rank):
    rng = np.random.default_rng([m, n, rank])
    w, what = weight(rng, n, 320, 4, 64)
    p = pool(rng, 7, n, 320, rank, scaled=rank != 48)
    for ids in (rng.integers(-1, 7, m), np.sort(rng.integers(-1, 7, m)), np.full(m, 6)):
        lora_check(w, what, rows(rng, m, 320), p, ids.astype(np.int32), f"rank {rank}")


@pytest.mark.parametrize("bits", WIDTHS)
@pytest.mark.parametrize("form", EXPERTS_32, ids=lambda f: "-".join(map(str, f)))
def test_experts_32_rows(form, bits):
    m, top_k, experts, inner, model = EXPERTS_32[form]
    rng = np.random.default_rng([inner, bits])
    ws, what = experts_of(rng, experts, inner, model, bits, 10 - bits, "64" if bits % 2 else "k")
    x = rows(rng, m, model)
    ids, w = routed(rng, m, experts, top_k)
    moe_check(ws, what, x, ids, w, "spread")
    moe_check(ws, what, x, np.full_like(ids, 3), w, "one expert")


@pytest.mark.parametrize("bits", WIDTHS)
@pytest.mark.parametrize("form", EXPERTS_1, ids=lambda f: "-".join(map(str, f)))
def test_experts_one_row(form, bits):
    m, top_k, experts, inner, model = EXPERTS_1[form]
    rng = np.random.default_rng([model, bits])
    ws, what = experts_of(rng, experts, inner, model, bits, 10 - bits, "k" if bits % 2 else "64")
    ids, w = routed(rng, m, experts, top_k)
    moe_check(ws, what, rows(rng, m, model), ids, w, "random")
