"""One row has no next one: its distance to it in the tensor that it is a view of is not
passed on, and not refused."""
import numpy as np
import pytest
import torch

from group_wise_bit_amd import qlin


@pytest.mark.parametrize("width", [64, 65, 100, 1000])
def test_pitch_of_one_row(width):
    t = torch.zeros(3, width)
    assert qlin._row_pitch(t[:1, :64]) == 64
    assert qlin._row_pitch(t[:2, :64]) == width
    assert qlin._row_pitch(t[:0, :64]) == 64


@pytest.mark.gpu
@pytest.mark.parametrize("extra", [1, 4, 7, 8])
def test_one_row_of_a_wider_tensor(extra):
    import rows_ref as rr
    from test_gpu_rows_lora import dev, pool, weight
    from test_gpu_rows_moe import experts_of, routed
    rng = np.random.default_rng(extra)
    w, what = weight(rng, 130, 192, 4, 64)
    p = pool(rng, 3, 130, 192, 16)
    x = rng.standard_normal((5, 192 + extra), dtype=np.float32).astype(np.float16)
    row = dev(x)[:1, :192]
    ids = np.array([2], np.int32)
    y, _ = qlin.gemm_lora(w, row, qlin.Adapters(*map(dev, p)), dev(ids))
    rr.check(y.cpu().numpy(), *rr.lora_ref(x[:1, :192], what, *p, ids), "adapters")
    ws, whats = experts_of(rng, 4, 128, 192, 4, 4)
    eids, wts = routed(rng, 1, 4, 2)
    y, _ = qlin.moe_mlp(*ws, row, dev(eids), dev(wts))
    rr.check(y.cpu().numpy(), *rr.moe_ref(x[:1, :192], *whats, eids, wts), "experts")
    logits = torch.randn(4, 8 + extra, device="cuda")[:1, :8]
    a, b = qlin.route(qlin.Router(8, 2), logits), qlin.route(qlin.Router(8, 2), logits.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
