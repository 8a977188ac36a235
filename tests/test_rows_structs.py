"""The cached C structures of routers, expert stacks and adapters: a tensor put in the place
of another is checked as one of a new object would be, whatever its address and size."""
import pytest
import torch

from group_wise_bit_amd import qlin


def test_router_bias():
    big = torch.zeros(128)
    r = qlin.Router(64, 2, bias=big[:64])
    assert r.c_struct() is r.c_struct()
    assert r.c_struct().bias == big.data_ptr()
    for other in (big[::2], big[:64].view(1, 64), big[:64].view(8, 8)):
        r.bias = other
        with pytest.raises(TypeError):
            r.c_struct()
    r.bias = big[64:]
    assert r.c_struct().bias == big.data_ptr() + 256
    r.bias = None
    assert not r.c_struct().bias
    r.top_k = 3
    assert r.c_struct().top_k == 3


def stack():
    e = 2 * qlin.meta_entries(128, 64, 64)
    return qlin.QExperts(2, 128, 64, 4, 64,
                         torch.zeros(2 * qlin.packed_bytes(128, 64, 4) // 4, dtype=torch.int32),
                         torch.zeros(e, dtype=torch.float16), torch.zeros(e, dtype=torch.uint8))


@pytest.mark.parametrize("field", ["data", "scale", "zero"])
def test_expert_stack(field):
    q = stack()
    q.c_struct()
    t = getattr(q, field)
    wide = torch.zeros(2 * t.numel(), dtype=t.dtype)
    setattr(q, field, wide[:t.numel()])
    assert getattr(q.c_struct(), field) == wide.data_ptr()
    setattr(q, field, wide[::2])                  # the same address, size and type
    with pytest.raises(ValueError):
        q.c_struct()


def test_adapters():
    w = stack().expert(0)
    a, b = torch.zeros(3, 64, 64).half(), torch.zeros(3, 128, 64).half()
    scale = torch.zeros(6)
    ad = qlin.Adapters(a, b, scale[:3])
    assert ad.c_struct(w) is ad.c_struct(w)
    ad.a = a.transpose(1, 2)                      # rank = k: the same shape too
    with pytest.raises(TypeError):
        ad.c_struct(w)
    ad.a = a
    ad.scale = scale[::2]
    with pytest.raises(TypeError):
        ad.c_struct(w)
    ad.scale = scale[3:]
    assert ad.c_struct(w).scale == scale.data_ptr() + 12
    square = qlin.QWeight(64, 64, 4, 64, qlin.FMT_PACKED, w.data, w.scale, w.zero)
    ad = qlin.Adapters(a, torch.zeros(3, 64, 64).half())
    ad.c_struct(square)
    ad.b = ad.b.transpose(1, 2)                   # n = rank
    with pytest.raises(TypeError):
        ad.c_struct(square)
