"""The cached workspaces on a GPU: a graph of a dense call and eager calls of larger
workspaces on its stream (the replays give the eager result and write to nothing else), and
threads that make row-wise calls on one stream."""
import threading

import numpy as np
import pytest
import torch

import rows_ref as rr
from group_wise_bit_amd import qlin
from test_gpu_rows_lora import dev, pool, weight
from test_gpu_rows_moe import experts_of, routed

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_graph_of_a_dense_call_and_growing_calls():
    rng = np.random.default_rng(1)
    w, what = weight(rng, 128, 8192, 4, 64)          # two tiles: split across work-groups
    big, _ = weight(rng, 1024, 8192, 4, 64)
    x = dev(rng.standard_normal((8, 8192), dtype=np.float32).astype(np.float16))
    ws, whats = experts_of(rng, 8, 512, 256, 4, 4)
    xe = rng.standard_normal((300, 256), dtype=np.float32).astype(np.float16)
    ids, we = routed(rng, 300, 8, 2)
    args = [dev(t) for t in (xe, ids, we)]
    ref, err = rr.moe_ref(xe, *whats, ids, we)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = qlin.gemm(w, x).clone()               # the stream's cached workspace
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = qlin.gemm(w, x)
    with torch.cuda.stream(side):
        y = qlin.moe_mlp(*ws, *args)[0]              # a larger workspace, eagerly
        qlin.gemm(big, x)                            # and a larger one of the dense calls
        # everything the allocator has to give is taken by tensors of one value
        fill = [torch.full((1 << 18,), 7, dtype=torch.uint8, device=DEV) for _ in range(200)]
    side.synchronize()
    rr.check(y.cpu().numpy(), ref, err, "experts")
    for _ in range(3):
        with torch.cuda.stream(side):
            graph.replay()
            again = qlin.moe_mlp(*ws, *args)[0]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(again, y)
        assert all((t == 7).all() for t in fill)


def test_threads_on_one_stream():
    """Four threads, each its own batches of experts and adapters, on the default stream."""
    rng = np.random.default_rng(2)
    ws, _ = experts_of(rng, 8, 512, 256, 4, 4)
    w, _ = weight(rng, 300, 256, 4, 64)
    ad = qlin.Adapters(*map(dev, pool(rng, 3, 300, 256, 64)))
    sets = []
    for m in (40, 90, 300, 420):
        x = dev(rng.standard_normal((m, 256), dtype=np.float32).astype(np.float16))
        ids, we = map(dev, routed(rng, m, 8, 2))
        slots = dev(rng.integers(-1, 3, m).astype(np.int32))
        sets.append((x, ids, we, slots))
    once = [(qlin.moe_mlp(*ws, *s[:3])[0], qlin.gemm_lora(w, s[0], ad, s[3])[0]) for s in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]

    def thread(i):
        for _ in range(30):
            got[i].append((qlin.moe_mlp(*ws, *sets[i][:3])[0],
                           qlin.gemm_lora(w, sets[i][0], ad, sets[i][3])[0]))
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(len(sets))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for want, have in zip(once, got):
        assert len(have) == 30
        assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in have)
