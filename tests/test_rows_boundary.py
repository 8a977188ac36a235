"""include/qlin_rows.h: exported symbols, host-side refusals of every entry
point (raised before any HIP call, so they run without a GPU), the workspace
queries, and the binding's own checks."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from group_wise_bit_amd import qlin

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlin_rows.h")
OK, NULL, SHAPE, BITS, GROUP, ALIGN, FORMAT, ALIAS, WORKSPACE, NODEV, HIP = range(11)
GB = 1 << 30
FAKE = 0x7F0000000000        # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return qlin.library()


def test_header_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(qlin_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(qlin.ROWS_EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


def router(**kw):
    d = dict(experts=64, top_k=8, score=0, groups=1, top_groups=1, group_top=1, renormalize=1,
             scale=1.0, bias=None)
    d.update(kw)
    return qlin.QlinRouterC(*[d[f] for f, _ in qlin.QlinRouterC._fields_])


def route(lib, r, logits=FAKE, m=4, ld=None, ids=FAKE + GB, weights=FAKE + 2 * GB):
    return lib.qlin_route(ctypes.byref(r) if r is not None else None, logits, m,
                          (r.experts if r is not None else 64) if ld is None else ld, ids, weights,
                          None)


def test_route_refusals(lib):
    assert route(lib, None) == NULL
    for kw in (dict(logits=None), dict(ids=None), dict(weights=None)):
        assert route(lib, router(), **kw) == NULL
    for kw in (dict(experts=0), dict(experts=513), dict(top_k=0), dict(top_k=33),
               dict(top_k=65, experts=64), dict(groups=0), dict(groups=3), dict(groups=65, experts=65),
               dict(groups=8, top_groups=0), dict(groups=8, top_groups=9), dict(group_top=0),
               dict(group_top=3), dict(groups=16, top_groups=1, top_k=5)):
        assert route(lib, router(**kw)) == SHAPE, kw
    assert route(lib, router(), m=-1) == SHAPE
    assert route(lib, router(), m=(1 << 20) + 1) == SHAPE
    assert route(lib, router(), ld=63) == SHAPE
    assert route(lib, router(score=2)) == FORMAT
    assert route(lib, router(renormalize=2)) == FORMAT
    assert route(lib, router(), logits=FAKE + 2) == ALIGN
    assert route(lib, router(bias=FAKE + 1)) == ALIGN
    assert route(lib, router(), ids=FAKE) == ALIAS
    assert route(lib, router(), weights=FAKE + GB + 64) == ALIAS
    assert route(lib, router(bias=FAKE + GB)) == ALIAS
    assert route(lib, router(), m=0, logits=None, ids=None, weights=None) == OK
    assert route(lib, router()) == NODEV or torch.cuda.is_available()


def weight(n, k, bits=4, group=64, at=0, **kw):
    d = dict(n=n, k=k, bits=bits, group=group, format=0, reserved=0, data=FAKE + (16 + at) * GB,
             ld=0, scale=FAKE + (17 + at) * GB, zero=FAKE + (18 + at) * GB)
    d.update(kw)
    return qlin.QlinWeightC(*[d[f] for f, _ in qlin.QlinWeightC._fields_])


def moe(lib, gate=None, up=None, down=None, experts=4, X=FAKE, m=3, ldx=128, ids=FAKE + GB,
        weights=FAKE + 2 * GB, top_k=2, Y=FAKE + 3 * GB, Y16=None, ldy=128, ws=FAKE + 4 * GB,
        wsb=None):
    gate = weight(192, 128) if gate is None else gate
    up = weight(192, 128, at=4) if up is None else up
    down = weight(128, 192, at=8) if down is None else down
    if wsb is None:
        wsb = lib.qlin_moe_mlp_workspace_bytes(ctypes.byref(gate), ctypes.byref(down), experts, m,
                                               top_k)
    return lib.qlin_moe_mlp(ctypes.byref(gate), ctypes.byref(up), ctypes.byref(down), experts, X,
                            m, ldx, ids, weights, top_k, Y, Y16, ldy, ws, wsb, None)


def test_moe_refusals(lib):
    assert moe(lib, up=weight(128, 128)) == SHAPE
    assert moe(lib, up=weight(192, 64)) == SHAPE
    assert moe(lib, down=weight(64, 192)) == SHAPE
    assert moe(lib, down=weight(128, 128)) == SHAPE
    assert moe(lib, gate=weight(100, 128), up=weight(100, 128)) == SHAPE   # inner not a block
    assert moe(lib, up=weight(192, 128, bits=3)) == FORMAT
    assert moe(lib, up=weight(192, 128, group=128)) == FORMAT
    assert moe(lib, gate=weight(192, 128, format=1, ld=128)) == FORMAT
    assert moe(lib, down=weight(128, 192, bits=9)) == BITS
    assert moe(lib, down=weight(128, 192, group=32)) == GROUP
    assert moe(lib, gate=weight(192, 128, data=None)) == NULL
    assert moe(lib, gate=weight(192, 128, scale=FAKE + 8)) == ALIGN
    for kw in (dict(experts=0), dict(experts=513), dict(top_k=0), dict(top_k=33), dict(m=-1),
               dict(m=(1 << 20) + 1), dict(ldx=120), dict(ldy=127)):
        assert moe(lib, wsb=1 << 40, **kw) == SHAPE, kw
    assert moe(lib, m=1 << 20, ldx=128, top_k=32, experts=64, wsb=1 << 50) in (ALIAS, SHAPE)
    assert moe(lib, ldx=132) == ALIGN
    for kw in (dict(X=None), dict(ids=None), dict(weights=None), dict(Y=None)):
        assert moe(lib, **kw) == NULL, kw
    for kw in (dict(X=FAKE + 2), dict(ids=FAKE + GB + 1), dict(weights=FAKE + 2 * GB + 2),
               dict(Y=FAKE + 3 * GB + 4), dict(Y16=FAKE + 9 * GB + 2), dict(ws=FAKE + 4 * GB + 8)):
        assert moe(lib, **kw) == ALIGN, kw
    assert moe(lib, ws=None) == WORKSPACE
    assert moe(lib, wsb=0) == WORKSPACE
    need = lib.qlin_moe_mlp_workspace_bytes(ctypes.byref(weight(192, 128)),
                                            ctypes.byref(weight(128, 192)), 4, 3, 2)
    assert need > 65536 and moe(lib, wsb=need - 1) == WORKSPACE
    for kw in (dict(Y=FAKE), dict(Y=FAKE + GB), dict(Y=FAKE + 2 * GB), dict(Y16=FAKE + 3 * GB),
               dict(Y=FAKE + 4 * GB), dict(Y=FAKE + 16 * GB), dict(Y=FAKE + 25 * GB),
               dict(ws=FAKE), dict(ws=FAKE + 20 * GB), dict(ws=FAKE + 26 * GB)):
        assert moe(lib, **kw) == ALIAS, kw
    # the last expert of a stack, not only the first
    one = qlin.packed_bytes(192, 128, 4)
    assert moe(lib, Y=FAKE + 16 * GB + 3 * one) == ALIAS
    assert moe(lib, m=0, X=None, ids=None, weights=None, Y=None, ws=None, wsb=0) == OK


def test_moe_workspace_query(lib):
    g, d = weight(192, 128), weight(128, 192)
    q = lib.qlin_moe_mlp_workspace_bytes
    assert q(ctypes.byref(g), ctypes.byref(d), 4, 0, 2) == 0
    assert q(ctypes.byref(g), ctypes.byref(g), 4, 3, 2) == 0
    assert q(None, ctypes.byref(d), 4, 3, 2) == 0
    assert q(ctypes.byref(g), None, 4, 3, 2) == 0
    assert q(ctypes.byref(g), ctypes.byref(d), 4, 1 << 20, 32) > 0
    assert q(ctypes.byref(g), ctypes.byref(d), 4, (1 << 20) + 1, 32) == 0


def adapters(**kw):
    d = dict(slots=5, rank=16, a=FAKE + 8 * GB, b=FAKE + 9 * GB, scale=None)
    d.update(kw)
    return qlin.QlinAdaptersC(*[d[f] for f, _ in qlin.QlinAdaptersC._fields_])


def lora(lib, w=None, ad=None, X=FAKE, m=3, ldx=128, ids=FAKE + GB, Y=FAKE + 3 * GB, Y16=None,
         ldy=200, ws=FAKE + 4 * GB, wsb=None):
    w = weight(200, 128) if w is None else w
    ad = adapters() if ad is None else ad
    if wsb is None:
        wsb = lib.qlin_gemm_lora_workspace_bytes(ctypes.byref(w), ctypes.byref(ad), m)
    return lib.qlin_gemm_lora(ctypes.byref(w), ctypes.byref(ad), X, m, ldx, ids, Y, Y16, ldy, ws,
                              wsb, None)


def test_lora_refusals(lib):
    assert lora(lib, w=weight(200, 100)) == SHAPE
    assert lora(lib, w=weight(200, 128, bits=16)) == BITS
    assert lora(lib, w=weight(200, 128, format=1, ld=128)) == FORMAT
    assert lora(lib, w=weight(200, 128, zero=None)) == NULL
    for kw in (dict(slots=0), dict(slots=513), dict(rank=0), dict(rank=4), dict(rank=12),
               dict(rank=136)):
        assert lora(lib, ad=adapters(**kw)) == SHAPE, kw
    for kw in (dict(m=-1), dict(m=(1 << 20) + 1), dict(ldx=64), dict(ldy=199)):
        assert lora(lib, wsb=1 << 40, **kw) == SHAPE, kw
    assert lora(lib, ldx=130) == ALIGN
    for kw in (dict(X=None), dict(ids=None), dict(Y=None), dict(ad=adapters(a=None)),
               dict(ad=adapters(b=None))):
        assert lora(lib, **kw) == NULL, kw
    for kw in (dict(X=FAKE + 8), dict(ids=FAKE + GB + 2), dict(Y=FAKE + 3 * GB + 8),
               dict(ad=adapters(a=FAKE + 8 * GB + 8)), dict(ad=adapters(b=FAKE + 9 * GB + 2)),
               dict(ad=adapters(scale=FAKE + 10 * GB + 1)), dict(ws=FAKE + 4 * GB + 4)):
        assert lora(lib, **kw) == ALIGN, kw
    assert lora(lib, ws=None) == WORKSPACE
    need = lib.qlin_gemm_lora_workspace_bytes(ctypes.byref(weight(200, 128)),
                                              ctypes.byref(adapters()), 3)
    assert need > 65536 and lora(lib, wsb=need - 1) == WORKSPACE
    for kw in (dict(Y=FAKE), dict(Y=FAKE + GB), dict(Y16=FAKE + 3 * GB), dict(Y=FAKE + 8 * GB),
               dict(Y=FAKE + 9 * GB), dict(Y=FAKE + 17 * GB), dict(Y=FAKE + 4 * GB),
               dict(ws=FAKE + 16 * GB), dict(ad=adapters(scale=FAKE + 3 * GB))):
        assert lora(lib, **kw) == ALIAS, kw
    assert lora(lib, m=0, X=None, ids=None, Y=None, ws=None, wsb=0) == OK
    q = lib.qlin_gemm_lora_workspace_bytes
    assert q(ctypes.byref(weight(200, 128)), ctypes.byref(adapters(rank=7)), 3) == 0
    assert q(ctypes.byref(weight(200, 128)), None, 3) == 0


def cpu_stack(count=3, n=128, k=64, bits=4):
    t = count * qlin.meta_entries(n, k, 64)
    return qlin.QExperts(count, n, k, bits, 64,
                         torch.zeros(count * qlin.packed_bytes(n, k, bits) // 4, dtype=torch.int32),
                         torch.zeros(t, dtype=torch.float16), torch.zeros(t, dtype=torch.uint8))


def test_binding_refuses_before_any_launch():
    r = qlin.Router(8, 2)
    for bad in (torch.zeros(4, 8, dtype=torch.float16), torch.zeros(4, 7), torch.zeros(8),
                torch.zeros(8, 4).t()):
        with pytest.raises(TypeError):
            qlin.route(r, bad)
    with pytest.raises(TypeError):
        qlin.route(r, torch.zeros(4, 8), ids=torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(TypeError):
        qlin.route(r, torch.zeros(4, 8), weights=torch.zeros(4, 3))
    with pytest.raises(TypeError):
        qlin.route(qlin.Router(8, 2, bias=torch.zeros(7)), torch.zeros(4, 8))
    with pytest.raises(ValueError):
        qlin.route(qlin.Router(8, 2, score="relu"), torch.zeros(4, 8))
    with pytest.raises(ValueError):
        qlin.route(r, torch.zeros(4, 8))                      # not on a GPU
    with pytest.raises(ValueError):
        qlin.route(qlin.Router(8, 2, bias=torch.zeros(8, device="meta")), torch.zeros(4, 8))

    g, u, d = cpu_stack(), cpu_stack(), cpu_stack(n=64, k=128)
    X, ids, w = (torch.zeros(5, 64, dtype=torch.float16), torch.zeros(5, 2, dtype=torch.int32),
                 torch.zeros(5, 2))
    with pytest.raises(TypeError):
        qlin.moe_mlp(g, u, d, X.float(), ids, w)
    with pytest.raises(TypeError):
        qlin.moe_mlp(g, u, d, X[:, :32], ids, w)
    with pytest.raises(TypeError):
        qlin.moe_mlp(g, u, d, X, ids.long(), w)
    with pytest.raises(TypeError):
        qlin.moe_mlp(g, u, d, X, ids[:4], w)
    with pytest.raises(TypeError):
        qlin.moe_mlp(g, u, d, X, ids, w.half())
    with pytest.raises(ValueError):
        qlin.moe_mlp(g, cpu_stack(count=2), d, X, ids, w)
    with pytest.raises(ValueError):
        qlin.moe_mlp(g, u, d, X, ids, w, want_y=False, want_y16=False)
    with pytest.raises(ValueError):
        qlin.moe_mlp(g, u, d, X, ids, w, Y=torch.zeros(5, 63))
    with pytest.raises(ValueError):
        qlin.moe_mlp(g, u, d, X, ids, w, Y=torch.zeros(5, 64), Y16=torch.zeros(5, 72).half())
    short = cpu_stack()
    short.data = short.data[:-1]
    with pytest.raises(ValueError):
        qlin.moe_mlp(short, u, d, X, ids, w)
    with pytest.raises(IndexError):
        g.expert(3)
    with pytest.raises(TypeError):
        qlin.quantize_experts(X, 4, 64)

    e = g.expert(0)
    ad = qlin.Adapters(torch.zeros(2, 8, 64).half(), torch.zeros(2, 128, 8).half())
    lid = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(TypeError):
        qlin.gemm_lora(e, X, ad, lid[:3])
    with pytest.raises(TypeError):
        qlin.gemm_lora(e, X, ad, lid.float())
    with pytest.raises(TypeError):
        qlin.gemm_lora(e, X, qlin.Adapters(ad.a, ad.b[:, :64]), lid)
    with pytest.raises(TypeError):
        qlin.gemm_lora(e, X, qlin.Adapters(ad.a.transpose(1, 2), ad.b), lid)
    with pytest.raises(TypeError):
        qlin.gemm_lora(e, X, qlin.Adapters(ad.a, ad.b, torch.zeros(3)), lid)
    with pytest.raises(ValueError):
        qlin.gemm_lora(e, X, ad, lid, Y=torch.zeros(4, 128))


def test_stack_views_cover_the_stack():
    s = cpu_stack(count=4, n=100, k=128, bits=5)
    s.data.copy_(torch.arange(s.data.numel(), dtype=torch.int32))
    got = torch.cat([s.expert(e).data for e in range(4)])
    assert torch.equal(got, s.data)
    assert all(s.expert(e).data.data_ptr() % 16 == 0 for e in range(4))
    assert s.expert(3).zero.numel() == qlin.meta_entries(100, 128, 64)
    assert np.prod(s.expert(1).scale.shape) == qlin.meta_entries(100, 128, 64)
