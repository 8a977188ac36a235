"""Calls of the row-wise entry points that pass every host check, with made-up addresses: they
are made only where no GPU is there to run them, and then end in QLIN_ERR_NO_DEVICE."""
import pytest
import torch

import conftest
import test_rows_boundary as tb
from group_wise_bit_amd import qlin


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_no_device():
    lib = qlin.library()
    assert tb.route(lib, tb.router()) == tb.NODEV
    assert tb.route(lib, tb.router(score=1, groups=8, top_groups=4, group_top=2)) == tb.NODEV
    assert tb.moe(lib) == tb.NODEV
    assert tb.moe(lib, m=300, Y16=tb.FAKE + 9 * tb.GB) == tb.NODEV
    assert tb.lora(lib) == tb.NODEV
    assert tb.lora(lib, m=300, Y16=tb.FAKE + 5 * tb.GB) == tb.NODEV


class Item:
    def __init__(self, nodeid):
        self.nodeid, self.marks = nodeid, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


@pytest.mark.parametrize("gpu", [False, True])
def test_made_up_addresses_stay_off_a_gpu(monkeypatch, gpu):
    """tests/test_rows_boundary.py::test_route_refusals ends with such a call."""
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    items = [Item("tests/test_rows_boundary.py::test_route_refusals"),
             Item("tests/test_rows_boundary.py::test_moe_refusals")]
    conftest.pytest_collection_modifyitems(items)
    assert items[0].marks == (["skip"] if gpu else []) and items[1].marks == []
