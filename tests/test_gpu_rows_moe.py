"""GPU parity of qlin_moe_mlp against the 64-bit reference, within the derived
bounds of rows_ref, at every width and over row counts from one to many rows
per expert; empty and padded rows, repeated experts, pitches, aliases of the
workspace, other streams, capture and replay."""
import numpy as np
import pytest
import torch

import oracle
import rows_ref as rr
from group_wise_bit_amd import qlin

pytestmark = pytest.mark.gpu
DEV = "cuda"


def stack(rng, count, n, k, bits, group):
    w, s, z, what = rr.packed_stack(rng, count, n, k, bits, group)
    return qlin.QExperts(count, n, k, bits, group, torch.from_numpy(w).to(DEV),
                         torch.from_numpy(s).to(DEV), torch.from_numpy(z).to(DEV)), what


def experts_of(rng, count, inner, model, bits, dbits, group="64"):
    gg, gd = (64, 64) if group == "64" else (model, inner)
    g, wg = stack(rng, count, inner, model, bits, gg)
    u, wu = stack(rng, count, inner, model, bits, gg)
    d, wd = stack(rng, count, model, inner, dbits, gd)
    return (g, u, d), (wg, wu, wd)


def routed(rng, m, experts, top_k):
    ids = np.stack([rng.permutation(experts)[:top_k] for _ in range(m)]).astype(np.int32) \
        if m else np.zeros((0, top_k), np.int32)
    w = rng.random((m, top_k), dtype=np.float32) + np.float32(0.05)
    return ids, (w / w.sum(1, keepdims=True)).astype(np.float32)


def call(ws, x, ids, w, **kw):
    y, y16 = qlin.moe_mlp(*ws, torch.from_numpy(x).to(DEV), torch.from_numpy(ids).to(DEV),
                          torch.from_numpy(w).to(DEV), **kw)
    torch.cuda.synchronize()
    return y, y16


def check(ws, what, x, ids, w, label):
    y, y16 = call(ws, x, ids, w)
    ref, err = rr.moe_ref(x, *what, ids, w)
    rr.check(y.cpu().numpy(), ref, err, label)
    rr.check_half(y16.cpu().numpy(), ref, err, label + " fp16")
    assert torch.equal(y.half(), y16), label
    return y


@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("group", ["64", "k"])
def test_every_width(bits, group):
    rng = np.random.default_rng([bits, len(group)])
    ws, what = experts_of(rng, 5, 192, 256, bits, {2: 8, 3: 4, 4: 2, 5: 7, 6: 3, 7: 6, 8: 5}[bits],
                          group)
    for m in (1, 9, 70):
        x = rng.standard_normal((m, 256), dtype=np.float32).astype(np.float16)
        ids, w = routed(rng, m, 5, 2)
        check(ws, what, x, ids, w, f"{bits} bits m={m}")


@pytest.mark.parametrize("m,experts,top_k,inner,model", [
    (1, 1, 1, 64, 64), (1, 8, 8, 128, 64), (2, 7, 3, 64, 192), (3, 40, 4, 128, 128),
    (31, 4, 1, 192, 64), (33, 2, 2, 64, 320), (64, 3, 1, 128, 128), (65, 1, 1, 64, 128),
    (127, 3, 2, 128, 64), (129, 2, 1, 192, 128), (200, 16, 4, 64, 64), (300, 2, 2, 128, 192),
    (257, 1, 1, 64, 64), (520, 3, 1, 64, 128)])
def test_row_counts(m, experts, top_k, inner, model):
    rng = np.random.default_rng([m, experts, inner])
    ws, what = experts_of(rng, experts, inner, model, 4, 4)
    x = rng.standard_normal((m, model), dtype=np.float32).astype(np.float16)
    ids, w = routed(rng, m, experts, top_k)
    check(ws, what, x, ids, w, "random")
    # every row to one expert (the same expert in all its slots)
    check(ws, what, x, np.full_like(ids, experts - 1), w, "one expert")


def test_long_k_and_many_experts():
    rng = np.random.default_rng(8)
    ws, what = experts_of(rng, 3, 1088, 1216, 3, 8)
    for m in (1, 5, 140):
        x = rng.standard_normal((m, 1216), dtype=np.float32).astype(np.float16)
        check(ws, what, x, *routed(rng, m, 3, 2), f"long m={m}")
    ws, what = experts_of(rng, 512, 64, 64, 4, 4)
    x = rng.standard_normal((150, 64), dtype=np.float32).astype(np.float16)
    check(ws, what, x, *routed(rng, 150, 512, 9), "512 experts")


@pytest.mark.parametrize("m", [1, 6, 150])
def test_ids_outside_and_empty_rows(m):
    rng = np.random.default_rng(m)
    ws, what = experts_of(rng, 4, 128, 128, 4, 4)
    x = rng.standard_normal((m, 128), dtype=np.float32).astype(np.float16)
    ids, w = routed(rng, m, 4, 3)
    ids[rng.random(ids.shape) < 0.4] = -1
    ids[0] = [-1, 4, 2 ** 31 - 1]
    if m > 2:
        ids[2] = -(2 ** 31)
    w[(ids < 0) | (ids >= 4)] = np.nan          # a dropped slot's weight is not read
    y = check(ws, what, x, ids, np.where(np.isnan(w), 0, w).astype(np.float32), "dropped")
    y2, _ = call(ws, x, ids, w)
    assert torch.equal(y, y2)
    assert (y[0] == 0).all()
    y, y16 = call(ws, x, np.full_like(ids, -1), w)
    assert (y == 0).all() and (y16 == 0).all()


@pytest.mark.parametrize("m", [3, 140])
def test_rows_do_not_mix(m):
    """A row that is not finite, or carries a weight that is not, leaves the others alone."""
    rng = np.random.default_rng(20 + m)
    ws, what = experts_of(rng, 3, 128, 192, 4, 4)
    x = rng.standard_normal((m, 192), dtype=np.float32).astype(np.float16)
    ids, w = routed(rng, m, 3, 2)
    good, _ = call(ws, x, ids, w)
    x2, w2 = x.copy(), w.copy()
    x2[1, 5], x2[1, 70] = np.inf, np.nan
    w2[2] = np.nan
    bad, _ = call(ws, x2, ids, w2)
    keep = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(good[keep], bad[keep])
    assert not torch.isfinite(bad[1]).any() and torch.isnan(bad[2]).all()


@pytest.mark.parametrize("m", [4, 133])
def test_pitches_outputs_and_workspaces(m):
    rng = np.random.default_rng(m)
    ws, what = experts_of(rng, 4, 128, 192, 5, 3)
    x = rng.standard_normal((m, 192), dtype=np.float32).astype(np.float16)
    ids, w = routed(rng, m, 4, 2)
    y, y16 = call(ws, x, ids, w)
    X = torch.zeros(m, 264, dtype=torch.float16, device=DEV)
    X[:, 64:256] = torch.from_numpy(x).to(DEV)
    Y = torch.full((m + 2, 201), 7.0, device=DEV)
    Y16 = torch.full((m + 2, 201), 7.0, device=DEV).half()
    args = (X[:, 64:256], torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV))
    qlin.moe_mlp(*ws, *args, Y=Y, Y16=Y16)
    assert torch.equal(Y[:m, :192], y) and torch.equal(Y16[:m, :192], y16)
    assert (Y[m:] == 7).all() and (Y[:, 192:] == 7).all()
    assert (Y16[m:] == 7).all() and (Y16[:, 192:] == 7).all()
    only, none = qlin.moe_mlp(*ws, *args, want_y16=False)
    assert none is None and torch.equal(only, y)
    none, only = qlin.moe_mlp(*ws, *args, want_y=False)
    assert none is None and torch.equal(only, y16)
    # a workspace of any contents; its first 64 KiB (the other calls' counters) stay
    g, d = ws[0].c_struct(), ws[2].c_struct()
    import ctypes
    need = qlin.library().qlin_moe_mlp_workspace_bytes(ctypes.byref(g), ctypes.byref(d), 4, m, 2)
    for fill in (0, 255, 127):
        mine = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        y2, _ = qlin.moe_mlp(*ws, *args, ws=mine[:need])
        assert torch.equal(y2, y)
        assert (mine[:65536] == fill).all() and (mine[need:] == fill).all()


def test_stack_equals_its_experts():
    """quantize_experts gives the stack of qlin_quantize's buffers; one expert alone
    agrees with the dense gate/up and down calls."""
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.standard_normal((3, 128, 64), dtype=np.float32) * 0.02).half().to(DEV)
    st = qlin.quantize_experts(w, 4, 64)
    for e in range(3):
        q, v = qlin.quantize(w[e].contiguous(), 4, 64), st.expert(e)
        assert torch.equal(q.data, v.data) and torch.equal(q.zero, v.zero)
        assert torch.equal(q.scale.view(torch.int16), v.scale.view(torch.int16))
    up, down = qlin.quantize_experts(w * 1.5, 4, 64), qlin.quantize_experts(
        torch.from_numpy(rng.standard_normal((3, 64, 128), dtype=np.float32) * 0.02).half().to(DEV), 4, "K")
    x = torch.randn(10, 64, device=DEV).half()
    ids = torch.full((10, 1), 2, dtype=torch.int32, device=DEV)
    y, _ = qlin.moe_mlp(st, up, down, x, ids, torch.ones(10, 1, device=DEV))
    _, h = qlin.gemm_swiglu(st.expert(2), up.expert(2), x)
    ref = qlin.gemm(down.expert(2), h)
    # the dense calls round each weight to fp16 (a half step of 2^-11 each way)
    assert float((y - ref).abs().max()) <= 4 * 2.0 ** -11 * float(ref.abs().max()) * 8


@pytest.mark.parametrize("m", [1, 7, 160])
def test_reruns_streams_and_order(m):
    rng = np.random.default_rng(m)
    ws, _ = experts_of(rng, 6, 192, 256, 4, 4)
    x = rng.standard_normal((m, 256), dtype=np.float32).astype(np.float16)
    ids, w = routed(rng, m, 6, 3)
    y, _ = call(ws, x, ids, w)
    for _ in range(3):
        assert torch.equal(call(ws, x, ids, w)[0], y)
    args = (torch.from_numpy(x).to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(4):
                outs.append(qlin.moe_mlp(*ws, *args)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)


@pytest.mark.parametrize("m", [1, 5, 150])
def test_capture_and_replay(m):
    rng = np.random.default_rng(m)
    ws, _ = experts_of(rng, 6, 128, 192, 4, 3)
    mk = lambda: (torch.from_numpy(rng.standard_normal((m, 192), dtype=np.float32)  # noqa: E731
                                   .astype(np.float16)).to(DEV),
                  *(torch.from_numpy(t).to(DEV) for t in routed(rng, m, 6, 2)))
    x, ids, w = mk()
    qlin.moe_mlp(*ws, x, ids, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, y16 = qlin.moe_mlp(*ws, x, ids, w)
    for _ in range(4):
        nx, nids, nw = mk()
        nids[torch.rand(nids.shape, device=DEV) < 0.2] = -1
        x.copy_(nx), ids.copy_(nids), w.copy_(nw)
        graph.replay()
        eager, eager16 = qlin.moe_mlp(*ws, x.clone(), ids.clone(), w.clone())
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(y16, eager16)


def test_empty_batch():
    rng = np.random.default_rng(1)
    ws, _ = experts_of(rng, 2, 64, 64, 4, 4)
    y, y16 = qlin.moe_mlp(*ws, torch.empty(0, 64, device=DEV).half(),
                          torch.empty(0, 2, dtype=torch.int32, device=DEV),
                          torch.empty(0, 2, device=DEV))
    assert y.shape == (0, 64) and y16.shape == (0, 64)


def test_wide_scales_stay_exact():
    """Masters near fp16's end: q - z is exact, the scale is applied in fp32."""
    rng = np.random.default_rng(6)
    w16 = (rng.choice([-1.0, 1.0], (1, 64, 64)) * 65000 * rng.random((1, 64, 64))).astype(np.float16)
    codes, s16, z = oracle.quantize(w16[0], 2, 64)
    what = oracle.dequantize(codes, s16, z, 64)[None]
    st = qlin.quantize_experts(torch.from_numpy(w16).to(DEV), 2, 64)
    small, wsm = stack(rng, 1, 64, 64, 4, 64)
    x = (rng.standard_normal((3, 64)) * 1e-3).astype(np.float16)
    ids, w = np.zeros((3, 1), np.int32), np.ones((3, 1), np.float32)
    check((small, small, st), (wsm, wsm, what), x, ids, w, "wide down")
