"""The sizes of the GPU tests take the work-group forms that the tests are named for (no GPU
needed): a moved threshold fails here until the sizes follow it."""
import ctypes

import pytest

import rows_forms as rf
import test_gpu_rows_halves as halves
import test_gpu_rows_instances as inst
from group_wise_bit_amd import qlin


def test_instances_of_the_32_row_form():
    forms = {rf.ksplit(g) for g in range(1, 5000)}
    assert forms == {(32, 8), (64, 8), (64, 4)}
    assert set(inst.ADAPTERS) == {(how, *f) for how in ("dots", "come", "ordered") for f in forms}
    assert set(inst.EXPERTS_32) == forms
    assert set(inst.EXPERTS_1) == {rf.gemv(i, g) for i in (1, 1000) for g in (1, 100000)}


@pytest.mark.parametrize("bits", inst.WIDTHS)
def test_sizes_by_form(bits):
    for (how, cols, waves), (m, n, rank) in inst.ADAPTERS.items():
        assert rf.lora(m, n, 64 * (2 + bits % 4), rank) == (32, how, (cols, waves)), (how, cols, waves)
    for m, n, rank in inst.ORDERED:
        assert rf.lora(m, n, 320, rank)[:2] == (32, "ordered")
    assert {rf.lora(m, n, 320, rank)[2] for m, n, rank in inst.ORDERED} == {(32, 8), (64, 8), (64, 4)}
    for form, size in inst.EXPERTS_32.items():
        assert rf.moe(*size, bits, 10 - bits) == (32, form, form), form
    for form, size in inst.EXPERTS_1.items():
        assert rf.moe(*size, bits, 10 - bits) == (1, form, form), form


def test_sizes_of_the_64_row_form():
    """Those of tests/test_gpu_rows_forms.py."""
    for bits in range(2, 9):
        assert rf.moe(660, 1, 16, 1088, 192, bits, 10 - bits)[0] == 64
        assert rf.lora(250, 9200, 64 * (1 + bits % 5), 16)[0] == 64
    for model in (64, 128, 256, 320, 448):
        assert rf.moe(700, 2, 8, 1024, model, 4, 3)[0] == 64
    for rank in (8, 24, 64, 72, 128):
        assert rf.lora(580, 4160, 576, rank)[0] == 64
    # rows over more than 4 GB take the 32-row form
    assert rf.moe(660, 1, 16, 1088, 128, 4, 4, ld=1 << 22)[0] == 32
    assert rf.lora(660, 4096, 128, 16)[0] == 64 and rf.lora(660, 4096, 128, 16, ld=1 << 22)[0] == 32


def test_sizes_of_the_tests_of_halves():
    forms = [rf.moe(*size, 4, 4) for size in halves.SIZES]
    assert [f[0] for f in forms] == [1, 1, 1, 32, 32, 32, 64]
    assert [f[2] for f in forms[:6]] == [(16, 8), (8, 8), (8, 16), (32, 8), (64, 8), (64, 4)]
    for m, experts, inner, height in ((2, 3, 128, 1), (60, 3, 128, 32), (660, 16, 1088, 64)):
        assert rf.moe(m, 1, experts, inner, 256, 4, 4)[0] == height


def packed(n, k, bits=4):
    fake = 0x7F0000000000
    return qlin.QlinWeightC(n, k, bits, 64, 0, 0, fake, 0, fake, fake)


def test_the_rules_are_the_library_s():
    """The workspace that the library asks for shows which form it takes: one row, grouped,
    ordered or not, and how A x is split."""
    q = qlin.library().qlin_moe_mlp_workspace_bytes
    for m in (1, 2, 15, 16, 17, 32, 33, 500, 4096, 4097, 9000):
        for top_k, experts, inner, model, bits in ((1, 4, 128, 192, 4), (2, 16, 1024, 2048, 8),
                                                   (8, 64, 1024, 2048, 4), (2, 8, 1792, 4096, 8)):
            got = q(ctypes.byref(packed(inner, model, bits)), ctypes.byref(packed(model, inner)),
                    experts, m, top_k)
            assert got == rf.moe_workspace(m, top_k, experts, inner, model, bits, 4), (m, top_k, inner)
    q = qlin.library().qlin_gemm_lora_workspace_bytes
    for m in (1, 40, 96, 160, 161, 333, 640, 1024, 1030, 2560, 8193):
        for n, k, slots, rank in ((200, 192, 6, 24), (4096, 4096, 8, 64), (896, 4864, 5, 8),
                                  (6144, 4096, 64, 32), (64, 128, 512, 128)):
            ad = qlin.QlinAdaptersC(slots, rank, 0x7F0000000000, 0x7F0000000000, None)
            got = q(ctypes.byref(packed(n, k)), ctypes.byref(ad), m)
            assert got == rf.lora_workspace(m, n, k, slots, rank), (m, n, k, rank)


def test_a_grid_too_large_is_refused():
    """A host check before those of the call's addresses and workspace: 2^25 rows of 8192
    columns, and at 32 rows of X further apart 2^22 rows; not 2^21 rows of them."""
    import test_rows_boundary as tb
    big = dict(gate=tb.weight(64, 8192), up=tb.weight(64, 8192, at=4), down=tb.weight(8192, 64, at=8),
               experts=64, m=1 << 20, ldx=8192, ldy=8192)
    for top_k in (32, 4):
        assert tb.moe(qlin.library(), top_k=top_k, wsb=0, **big) == tb.SHAPE
    assert tb.moe(qlin.library(), top_k=2, wsb=0, **big) == tb.WORKSPACE
