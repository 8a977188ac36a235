"""The binding's cached workspaces: what a graph has recorded is never given back to the
allocator, and the row-wise calls' growing buffer is not the one that graphs of the other
calls record.  On the CPU, with the stream, its capture state and the library's calls
stood in for."""
import gc
import weakref

import pytest
import torch

from group_wise_bit_amd import qlin

CPU = torch.device("cpu")


@pytest.fixture
def stream(monkeypatch):
    """The state of the stream that the binding sees: its handle and whether it captures."""
    state = {"handle": 7, "capturing": False}
    monkeypatch.setattr(qlin, "_WS", {})
    monkeypatch.setattr(qlin, "_stream", lambda: state["handle"])
    monkeypatch.setattr(qlin, "_capturing", lambda: state["capturing"])
    monkeypatch.setattr(qlin, "_launch", lambda dev, call: call(state["handle"]))
    for name in ("_ROWS_WS", "_WS_RECORDED"):
        if hasattr(qlin, name):
            monkeypatch.setattr(qlin, name, type(getattr(qlin, name))())
    return state


def rows_call(need, seen):
    """A row-wise call of the given need, as _with_workspace makes it."""
    def call(ptr, size, stream):
        if size < need:
            return 8
        seen.append((ptr, size))
        return 0
    qlin._with_workspace("auto", CPU, lambda: need, call, "rows")


def test_recorded_buffer_outlives_a_larger_call(stream):
    qlin.workspace(100, CPU)                      # a warm-up call
    stream["capturing"] = True
    ref = weakref.ref(qlin.workspace(80, CPU))    # recorded by the graph
    stream["capturing"] = False
    assert qlin.workspace(10000, CPU).numel() == 10000
    gc.collect()
    assert ref() is not None and ref().numel() == 100


def test_unrecorded_buffer_is_replaced(stream):
    ref = weakref.ref(qlin.workspace(100, CPU))
    qlin.workspace(10000, CPU)
    gc.collect()
    assert ref() is None


def test_recorded_once(stream):
    stream["capturing"] = True
    for _ in range(3):
        qlin.workspace(64, CPU)
    assert len(qlin._WS_RECORDED) == 1


def test_row_wise_calls_leave_the_other_calls_buffer(stream):
    first = qlin.workspace(100, CPU)
    seen = []
    rows_call(5000, seen)
    assert qlin.workspace(100, CPU) is first
    assert seen[0][0] != first.data_ptr()


def test_row_wise_buffer_grows_and_is_kept(stream):
    seen = []
    for need in (500, 5000, 500, 5001):
        rows_call(need, seen)
    assert [size for _, size in seen] == [500, 5000, 5000, 5001]
    assert seen[1][0] == seen[2][0]
    stream["handle"] = 8
    rows_call(500, seen)
    assert seen[-1][1] == 500 and seen[-1][0] != seen[-2][0]


def test_row_wise_capture_takes_a_buffer_of_its_own(stream):
    seen = []
    rows_call(500, seen)
    stream["capturing"] = True
    rows_call(400, seen)
    stream["capturing"] = False
    rows_call(500, seen)
    assert seen[1][1] == 400 and seen[2] == seen[0]


def test_no_workspace_for_an_empty_call(stream):
    assert qlin.workspace(0, CPU) is None
    seen = []
    rows_call(0, seen)
    assert seen == [(None, 0)] or seen[0][1] == 0
