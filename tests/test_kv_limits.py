"""include/qlin_kv.h: the largest calls that are taken and the least that a grid's limit refuses."""
import ctypes

import pytest
import torch

from group_wise_bit_amd import qlin
from test_kv_boundary import FAKE, GB, NODEV, SHAPE, WORKSPACE, attend, cache, read, seqs, write

TB = 1 << 40
FAR = dict(K=FAKE + TB, V=FAKE + 2 * TB, ldk=65536, ldv=65536)


@pytest.fixture(scope="module")
def lib():
    return qlin.library()


@pytest.mark.parametrize("heads,ok", [(255, True), (256, False), (1024, False)])
def test_sequences_times_heads(lib, heads, ok):
    """seqs * heads < 2^24 (a call that is taken is one that lacks its workspace here)."""
    c, s = cache(kv_heads=1), seqs(seqs=65536, width=40, ld=40)
    kw = dict(ldq=heads * 64, ldo=heads * 64, heads=heads, Q=FAKE + TB, O=FAKE + 2 * TB)
    assert attend(lib, c, s, ws=None, **kw) == (WORKSPACE if ok else SHAPE)
    if not ok:
        least = seqs(seqs=(1 << 24) // heads, width=40, ld=40)
        most = seqs(seqs=(1 << 24) // heads - 1, width=40, ld=40)
        assert attend(lib, c, least, ws=None, **kw) == SHAPE
        assert attend(lib, c, most, ws=None, **kw) == WORKSPACE
    assert lib.qlin_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(s), heads) > 65536


def least_refused(call, lib, c, starts):
    """Sequences of one row each for which the header's product reaches 2^24."""
    parts = -(-c.kv_heads * (2 + c.head_dim // 64) // 4)
    tiles = -(-(1 << 24) // parts)
    if starts is None:
        return tiles, tiles
    n = next(n for n in range(1, 65537) if (n // 32 + 2 * n) * parts >= 1 << 24)
    return n, n


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kv_heads,head_dim", [(256, 256), (256, 128), (250, 256)])
@pytest.mark.parametrize("starts", [None, FAKE + 5 * GB])
def test_rows_times_parts(lib, call, kv_heads, head_dim, starts):
    c = cache(kv_heads=kv_heads, head_dim=head_dim, pages=1, k_bits=4, v_bits=4)
    n, m = least_refused(call, lib, c, starts)
    assert n <= 65536
    assert call(lib, c, seqs(seqs=n, width=1, ld=1), m=m, starts=starts, **FAR) == SHAPE
    if not torch.cuda.is_available():            # (made-up addresses)
        assert call(lib, c, seqs(seqs=n - 1, width=1, ld=1), m=n - 1, starts=starts, **FAR) == NODEV
