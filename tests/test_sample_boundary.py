"""include/qlin_sample.h: exported symbols, host-side refusals (raised before any HIP call, so they
run without a GPU), the binding's own checks, and the reference itself on small rows."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import sample_ref as sr
from group_wise_bit_amd import qlin

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlin_sample.h")
OK, NULL, SHAPE, BITS, GROUP, ALIGN, FORMAT, ALIAS, WORKSPACE, NODEV, HIP = range(11)
GB = 1 << 30
FAKE = 0x7F0000000000        # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return qlin.library()


def test_header_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(qlin_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(qlin.SAMPLE_EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


def sample(lib, s=(FAKE, FAKE + GB, FAKE + 2 * GB, FAKE + 3 * GB), logits=FAKE + 4 * GB, m=3,
           vocab=100, ld=100, u=FAKE + 5 * GB, ids=FAKE + 6 * GB, probs=FAKE + 7 * GB,
           ws=FAKE + 8 * GB, wsb=None):
    wsb = lib.qlin_sample_workspace_bytes(m, vocab) if wsb is None else wsb
    c = None if s is None else ctypes.byref(qlin.QlinSamplingC(*s))
    return lib.qlin_sample(c, logits, m, vocab, ld, u, ids, probs, ws, wsb, None)


def test_refusals(lib):
    assert sample(lib, s=None) == NULL
    for kw in (dict(logits=None), dict(u=None), dict(ids=None)):
        assert sample(lib, **kw) == NULL, kw
    for kw in (dict(m=-1), dict(m=(1 << 20) + 1), dict(vocab=0), dict(vocab=(1 << 18) + 1, ld=1 << 20),
               dict(ld=99)):
        assert sample(lib, wsb=1 << 40, **kw) == SHAPE, kw
    for i in range(4):
        s = [None] * 4
        s[i] = FAKE + 2
        assert sample(lib, s=s) == ALIGN
        s[i] = FAKE + 6 * GB + 8
        assert sample(lib, s=s) == ALIAS
    for kw in (dict(logits=FAKE + 1), dict(u=FAKE + 2), dict(ids=FAKE + 3), dict(probs=FAKE + 2),
               dict(ws=FAKE + 8 * GB + 8)):
        assert sample(lib, **kw) == ALIGN, kw
    for kw in (dict(ids=FAKE + 4 * GB + 1196), dict(probs=FAKE + 5 * GB), dict(ids=FAKE + 7 * GB + 4),
               dict(ws=FAKE + 4 * GB), dict(probs=FAKE + 8 * GB + 16)):
        assert sample(lib, **kw) == ALIAS, kw
    assert sample(lib, ws=None) == WORKSPACE
    need = lib.qlin_sample_workspace_bytes(3, 100)
    assert need >= 65536 and sample(lib, wsb=need - 1) == WORKSPACE
    assert sample(lib, m=0, logits=None, u=None, ids=None) == OK
    for bad in ((0, 5), (-1, 5), ((1 << 20) + 1, 5), (5, 0), (5, (1 << 18) + 1)):
        assert lib.qlin_sample_workspace_bytes(*bad) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")
def test_no_device(lib):
    assert sample(lib) == NODEV
    assert sample(lib, s=(None,) * 4, probs=None) == NODEV


def test_binding_refusals():
    x, u = torch.zeros(3, 50), torch.zeros(3)
    good = qlin.Sampling()
    for bad in (x.half(), x[0], x.t().contiguous().t()):
        with pytest.raises(TypeError):
            qlin.sample(good, bad, u)
    for bad in (u.double(), u[:2], torch.zeros(6)[::2], None):
        with pytest.raises(TypeError):
            qlin.sample(good, x, bad)
    for kw in (dict(temperature=u.double()), dict(top_k=u), dict(top_p=u[:2]),
               dict(min_p=torch.zeros(3, dtype=torch.int32)), dict(top_k=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            qlin.sample(qlin.Sampling(**kw), x, u)
    with pytest.raises(TypeError):
        qlin.sample(good, x, u, ids=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        qlin.sample(good, x, u, probs=torch.zeros(4))
    with pytest.raises(ValueError, match="on a GPU"):
        qlin.sample(good, x, u)
    # the settings of one batch do not pass for another's
    s = qlin.Sampling(temperature=u)
    s.c_struct(3)
    with pytest.raises(TypeError):
        s.c_struct(2)


def test_reference():
    row = np.log(np.array([1, 8, 4, 2, 1], np.float64)).astype(np.float32)
    ids = [sr.sample_row(row, u)[0] for u in (0.0, 0.05, 0.07, 0.5, 0.57, 0.8, 0.9, 0.95)]
    assert ids == [0, 0, 1, 1, 2, 2, 3, 4]
    assert list(sr.kept_tokens(row, 1, 3, 1, 0)[0]) == [1, 2, 3]
    assert list(sr.kept_tokens(row, 1, 4, 1, 0)[0]) == [1, 2, 3, 0]      # equal ones by index
    assert list(sr.kept_tokens(row, 1, 0, 0.7, 0)[0]) == [1, 2]
    assert list(sr.kept_tokens(row, 1, 2, 0.7, 0)[0]) == [1, 2]          # of the two's mass
    assert list(sr.kept_tokens(row, 1, 2, 0.6, 0)[0]) == [1]
    assert list(sr.kept_tokens(row, 1, 0, 1, 0.2)[0]) == [1, 2, 3]
    assert sr.sample_row(row, 0.9, t=0)[0] == 1 and sr.sample_row(row, 0.9, k=1)[0] == 1
    assert sr.sample_row(np.full(3, -np.inf, np.float32), 0.5) == (-1, 0.0, 1.0)
    assert sr.sample_row(row, 1.0)[0] == 4 and sr.sample_row(row, -1.0)[0] == 0
