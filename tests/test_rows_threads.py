"""Threads of a program that make row-wise calls on one stream: a call's launches share the
stream's workspace, so another's do not come between them.  On the CPU, with the library's
calls stood in for."""
import threading
import time

import torch

from group_wise_bit_amd import qlin

CPU = torch.device("cpu")


def test_calls_on_one_stream_do_not_interleave(monkeypatch):
    monkeypatch.setattr(qlin, "_ROWS_WS", {})
    monkeypatch.setattr(qlin, "_capturing", lambda: False)
    monkeypatch.setattr(qlin, "_launch", lambda dev, call: call(7))
    launches, start = [], threading.Barrier(4)

    def call(name, need):
        def launch(ptr, size, stream):
            if size < need:
                return 8
            for step in range(3):               # the launches of one call, the GIL given up between
                launches.append((name, ptr))
                time.sleep(0.002)
            return 0
        return launch

    def thread(name):
        start.wait()
        for i in range(5):
            qlin._with_workspace("auto", CPU, lambda: 100 * (i + 1), call(name, 100 * (i + 1)), "rows")
    threads = [threading.Thread(target=thread, args=(n,)) for n in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(launches) == 60
    for i in range(0, 60, 3):
        assert launches[i] == launches[i + 1] == launches[i + 2]


def test_a_refused_call_leaves_the_others_free(monkeypatch):
    monkeypatch.setattr(qlin, "_ROWS_WS", {})
    monkeypatch.setattr(qlin, "_capturing", lambda: False)
    monkeypatch.setattr(qlin, "_launch", lambda dev, call: call(7))
    for _ in range(2):
        try:
            qlin._with_workspace("auto", CPU, lambda: 1, lambda p, b, s: 2, "rows")
        except qlin.QlinError as e:
            assert e.status == 2
        try:
            qlin._with_workspace("auto", CPU, lambda: 1, lambda p, b, s: 1 // 0, "rows")
        except ZeroDivisionError:
            pass
    qlin._with_workspace("auto", CPU, lambda: 1, lambda p, b, s: 0, "rows")
