"""A graph of a dense call on a stream, and eager calls of larger workspaces on it: the
graph's replays give the eager result and write to nothing else."""
import numpy as np
import pytest
import torch

import rows_ref as rr
from group_wise_bit_amd import qlin
from test_gpu_rows_lora import dev, weight
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
