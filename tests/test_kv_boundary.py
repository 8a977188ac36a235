"""include/qlin_kv.h: exported symbols, host-side refusals of every entry point (raised before any
HIP call, so they run without a GPU), the size queries, and the binding's own checks."""
import ctypes
import os
import re

import pytest
import torch

import kv_ref as kr
from group_wise_bit_amd import qlin

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlin_kv.h")
OK, NULL, SHAPE, BITS, GROUP, ALIGN, FORMAT, ALIAS, WORKSPACE, NODEV, HIP = range(11)
GB = 1 << 30
FAKE = 0x7F0000000000        # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return qlin.library()


def test_header_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(qlin_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(qlin.KV_EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


def test_page_bytes(lib):
    for d in (64, 128, 256):
        for page in (32, 64, 128, 256):
            for kb in (4, 8, 16):
                for vb in (4, 8, 16):
                    assert lib.qlin_kv_page_bytes(d, page, kb, vb) == \
                        page // 32 * kr.tile_bytes(d, kb, vb)
    for bad in ((96, 64, 4, 4), (128, 48, 4, 4), (128, 512, 4, 4), (128, 64, 3, 4), (128, 64, 4, 5),
                (0, 0, 0, 0)):
        assert lib.qlin_kv_page_bytes(*bad) == 0


def test_reference_layout_is_one_to_one():
    """Every bit of a tile's codes belongs to one code, every scale and zero to one group."""
    for d in (64, 256):
        for kb, vb in ((4, 8), (16, 4), (8, 16)):
            used = []
            for (code, scale, zero), bits in zip(kr.places(d, kb, vb), (kb, vb)):
                byte, bit = code
                for i in range(bits):
                    used.append((byte * 8 + bit + i).ravel())
                if bits < 16:
                    for i in range(16):
                        used.append((scale * 8 + i).ravel())
                    for i in range(8):
                        used.append((zero * 8 + i).ravel())
            import numpy as np
            used = np.sort(np.concatenate(used))
            assert np.array_equal(used, np.arange(8 * kr.tile_bytes(d, kb, vb)))


def cache(**kw):
    d = dict(pages=8, kv_heads=2, head_dim=64, page=32, k_bits=4, v_bits=8, data=FAKE)
    d.update(kw)
    return qlin.QlinKvCacheC(*[d[f] for f, _ in qlin.QlinKvCacheC._fields_])


def seqs(**kw):
    d = dict(seqs=3, width=4, table=FAKE + GB, ld=4, lengths=FAKE + 2 * GB)
    d.update(kw)
    return qlin.QlinKvSeqsC(*[d[f] for f, _ in qlin.QlinKvSeqsC._fields_])


def write(lib, c=None, s=None, K=FAKE + 3 * GB, ldk=128, V=FAKE + 4 * GB, ldv=128, m=5,
          starts=FAKE + 5 * GB):
    c, s = c or cache(), s or seqs()
    return lib.qlin_kv_write(ctypes.byref(c), K, ldk, V, ldv, m, ctypes.byref(s), starts, None)


def read(lib, c=None, s=None, K=FAKE + 3 * GB, ldk=128, V=FAKE + 4 * GB, ldv=128, m=5,
         starts=FAKE + 5 * GB, wide=0):
    c, s = c or cache(), s or seqs()
    return lib.qlin_kv_read(ctypes.byref(c), ctypes.byref(s), starts, m, K, ldk, V, ldv, wide, None)


def attend(lib, c=None, s=None, Q=FAKE + 3 * GB, ldq=256, heads=4, scale=0.125, window=0,
           O=FAKE + 4 * GB, O16=None, ldo=256, lse=None, ws=FAKE + 5 * GB, wsb=None):
    c, s = c or cache(), s or seqs()
    if wsb is None:
        wsb = lib.qlin_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(s), heads)
    return lib.qlin_kv_attention(ctypes.byref(c), ctypes.byref(s), Q, ldq, heads, scale, window, O,
                                 O16, ldo, lse, ws, wsb, None)


@pytest.mark.parametrize("call", [write, read, attend])
def test_refusals_of_caches_and_sequences(lib, call):
    for kw in (dict(k_bits=3), dict(v_bits=0), dict(k_bits=2), dict(v_bits=32)):
        assert call(lib, cache(**kw)) == BITS, kw
    for kw in (dict(pages=0), dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=80),
               dict(page=16), dict(page=48)):
        assert call(lib, cache(**kw)) == SHAPE, kw
    for kw in (dict(seqs=-1), dict(seqs=65537), dict(width=0), dict(width=1 << 23, ld=1 << 23),
               dict(ld=3)):
        assert call(lib, None, seqs(**kw)) == SHAPE, kw
    assert call(lib, cache(data=None)) == NULL
    assert call(lib, None, seqs(table=None)) == NULL
    assert call(lib, None, seqs(lengths=None)) == NULL
    assert call(lib, cache(data=FAKE + 8)) == ALIGN
    assert call(lib, None, seqs(table=FAKE + GB + 2)) == ALIGN
    assert call(lib, None, seqs(lengths=FAKE + GB + 1)) == ALIGN
    assert call(lib, cache(data=None), seqs(seqs=0, table=None, lengths=None)) == OK


@pytest.mark.parametrize("call", [write, read])
def test_refusals_of_rows(lib, call):
    for kw in (dict(m=-1), dict(m=(1 << 20) + 1), dict(ldk=120), dict(ldv=64), dict(m=2, starts=None)):
        assert call(lib, **kw) == SHAPE, kw
    for kw in (dict(ldk=132), dict(ldv=129), dict(K=FAKE + 3 * GB + 8), dict(V=FAKE + 4 * GB + 2),
               dict(starts=FAKE + 5 * GB + 2)):
        assert call(lib, **kw) == ALIGN, kw
    for kw in (dict(K=None), dict(V=None)):
        assert call(lib, **kw) == NULL, kw
    assert call(lib, m=0, K=None, V=None, c=cache(data=None)) == OK
    # the least grid that is refused: threads are counted in 32 bits
    big = dict(c=cache(kv_heads=256, head_dim=256, pages=1, k_bits=16, v_bits=16),
               ldk=65536, ldv=65536, s=seqs(seqs=65536, width=1))
    assert call(lib, m=1 << 20, K=FAKE + (1 << 42), V=FAKE + (1 << 41), **big) == SHAPE


def test_refusals_of_overlaps(lib):
    assert write(lib, K=FAKE + 64) == ALIAS
    assert write(lib, V=FAKE + 64) == ALIAS
    assert write(lib, s=seqs(table=FAKE + 128)) == ALIAS
    assert write(lib, s=seqs(lengths=FAKE + 128)) == ALIAS
    assert write(lib, starts=FAKE + 128) == ALIAS
    for kw in (dict(K=FAKE), dict(V=FAKE + 16), dict(K=FAKE + GB), dict(V=FAKE + 2 * GB),
               dict(K=FAKE + 5 * GB), dict(K=FAKE + 4 * GB), dict(K=FAKE + 4 * GB + 128),
               dict(K=FAKE + 4 * GB + 240, ldk=256, ldv=256),
               dict(K=FAKE + 4 * GB + 272, ldk=256, ldv=256),
               dict(K=FAKE + 4 * GB + 256, ldk=256, ldv=264)):
        assert read(lib, **kw) == ALIAS, kw
    for kw in (dict(O=FAKE), dict(O16=FAKE + 64), dict(lse=FAKE + 3 * GB), dict(O=FAKE + 3 * GB),
               dict(O=FAKE + GB), dict(lse=FAKE + 2 * GB), dict(O16=FAKE + 4 * GB),
               dict(lse=FAKE + 4 * GB), dict(ws=FAKE), dict(ws=FAKE + 4 * GB), dict(O16=FAKE + 5 * GB)):
        assert attend(lib, **kw) == ALIAS, kw


def test_read_wide(lib):
    assert read(lib, wide=2) == FORMAT


def test_refusals_of_attention(lib):
    for kw in (dict(heads=0), dict(heads=3), dict(heads=1026), dict(ldq=248), dict(ldo=192),
               dict(window=-1)):
        assert attend(lib, wsb=1 << 40, **kw) == SHAPE, kw
    for kw in (dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attend(lib, **kw) == FORMAT, kw
    for kw in (dict(ldq=260), dict(ldo=257), dict(Q=FAKE + 3 * GB + 8), dict(O=FAKE + 4 * GB + 4),
               dict(O16=FAKE + 8 * GB + 2), dict(lse=FAKE + 8 * GB + 2), dict(ws=FAKE + 5 * GB + 8)):
        assert attend(lib, **kw) == ALIGN, kw
    assert attend(lib, Q=None) == NULL
    assert attend(lib, O=None) == NULL
    assert attend(lib, ws=None) == WORKSPACE
    need = lib.qlin_kv_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(seqs()), 4)
    assert need > 65536 and attend(lib, wsb=need - 1) == WORKSPACE
    for c, s, heads in ((cache(page=16), seqs(), 4), (cache(), seqs(width=0), 4), (cache(), seqs(), 5)):
        assert lib.qlin_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(s), heads) == 0
    # the workspace does not grow with the sequences beyond what the chip holds at once
    large = lib.qlin_kv_attention_workspace_bytes(
        ctypes.byref(cache(kv_heads=8, head_dim=256)), ctypes.byref(seqs(seqs=4096, width=4096, ld=4096)), 128)
    assert large <= 64 << 20


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")
def test_no_device(lib):
    assert write(lib) == NODEV and write(lib, starts=None, m=3) == NODEV
    assert read(lib) == NODEV and read(lib, wide=1) == NODEV
    assert read(lib, K=FAKE + 4 * GB + 256, ldk=256, ldv=256) == NODEV      # columns of one matrix
    assert attend(lib) == NODEV and attend(lib, O16=FAKE + 8 * GB, lse=FAKE + 9 * GB) == NODEV


def binding():
    c = qlin.kv_cache(4, 2, 64, 32, 4, 8, device="cpu")
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    return c, x, torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)


def test_binding_refusals():
    c, x, table, lengths = binding()
    starts = torch.zeros(4, dtype=torch.int32)
    for bad in (x.float(), x[:, :1], x[..., :32], x[0]):
        with pytest.raises((TypeError, ValueError)):
            qlin.kv_write(c, bad, x, table, lengths)
        with pytest.raises((TypeError, ValueError)):
            qlin.kv_write(c, x, bad, table, lengths)
    with pytest.raises(ValueError, match="strides"):
        qlin.kv_write(c, x.transpose(0, 1).contiguous().transpose(0, 1), x, table, lengths)
    with pytest.raises(ValueError, match="rows"):
        qlin.kv_write(c, x, x[:2], table, lengths)
    for t, l, s in ((table.long(), lengths, None), (table[0], lengths, None),
                    (table, lengths.long(), None), (table, lengths[:2], None),
                    (table, lengths, starts[:3]), (table, lengths, starts.long()),
                    (table.t().contiguous().t(), lengths, None)):
        with pytest.raises((TypeError, ValueError)):
            qlin.kv_write(c, x, x, t, l, starts=s)
        with pytest.raises((TypeError, ValueError)):
            qlin.kv_read(c, t, l, starts=s, rows=3)
    with pytest.raises(ValueError, match="rows must be given"):
        qlin.kv_read(c, table, lengths, starts=starts)
    with pytest.raises(TypeError, match="dtype"):
        qlin.kv_read(c, table, lengths, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        qlin.kv_read(c, table, lengths, K=x.float())
    with pytest.raises(ValueError, match="3 rows"):
        qlin.kv_read(c, table, lengths, K=x, V=x[:2])
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    for bad in (q.float(), q[0], q[..., :32]):
        with pytest.raises(TypeError):
            qlin.kv_attention(c, bad, table, lengths)
    with pytest.raises(ValueError, match="sequences"):
        qlin.kv_attention(c, q[:2], table, lengths)
    with pytest.raises(TypeError):
        qlin.kv_attention(c, q, table, lengths, O=torch.zeros(3, 4, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="row stride"):
        qlin.kv_attention(c, q, table, lengths, O=torch.zeros(3, 4, 64), O16=torch.zeros(
            3, 5, 64, dtype=torch.float16)[:, :4])
    with pytest.raises(TypeError):
        qlin.kv_attention(c, q, table, lengths, lse=torch.zeros(3, 5))
    with pytest.raises(ValueError, match="on a GPU"):
        qlin.kv_write(c, x, x, table, lengths)
    with pytest.raises(ValueError, match="on a GPU"):
        qlin.kv_attention(c, q, table, lengths)


def test_binding_refuses_caches():
    for kw in (dict(head_dim=80), dict(page_size=16), dict(k_bits=5), dict(v_bits=2)):
        with pytest.raises(ValueError, match="no cache layout"):
            qlin.kv_cache(**{**dict(pages=4, kv_heads=2, head_dim=64, device="cpu"), **kw})
    good = qlin.kv_cache(4, 2, 64, 32, 4, 8, device="cpu")
    for data in (good.data[:, :1], good.data[..., :-1], good.data.int(), good.data[0],
                 good.data.transpose(0, 1)):
        with pytest.raises(TypeError):
            qlin.KVCache(data, 2, 64, 32, 4, 8).c_struct()
    # another tensor in its place is looked at again
    good.c_struct()
    good.data = good.data[..., :-16].contiguous()
    with pytest.raises(TypeError):
        good.c_struct()


def test_binding_refuses_windows():
    """A window that 32 bits do not hold would come to another one's result."""
    c, _, table, lengths = binding()
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    for window in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="window"):
            qlin.kv_attention(c, q, table, lengths, window=window)
