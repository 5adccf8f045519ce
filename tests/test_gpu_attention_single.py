"""Attention of one new token per sequence over head rows (the kernel of every
decode step with up to 16 query heads to a key head) against the 64-bit form."""
import pytest
import torch

import position_independent_mla_gb300 as kv
from _serve import Batch, value64

pytestmark = pytest.mark.gpu


def requantise(b, change):
    """The pool's rows (values, keys; float64 [layers][slots][heads][128]) with `change`
    made to them in place, quantised again."""
    p = b.pool
    rows = [value64(p.copy, p.copy_scale).unflatten(-1, (-1, 128)),
            value64(p.rot, p.rot_scale).unflatten(-1, (-1, 128))]
    change(*rows)
    copy, rot = (x.flatten(-2).to(torch.bfloat16).contiguous() for x in rows)
    slots = copy.shape[1]
    src = kv.pool_desc(copy, rot, 1, b.h, 10000.0)
    ws = kv.quant_workspace(p.desc)
    kv.kv_quantize(src, None, p.desc, 0, slots,
                   torch.arange(slots, dtype=torch.int32, device="cuda"), ws)
    assert kv.kv_get_device_status(ws) == kv.KV_OK
    return b


SINGLE = [(1, 300), (1, 1500), (1, 64), (1, 1)]


@pytest.mark.parametrize("keys", [1.0, 0.0])
@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
def test_the_sum_does_not_depend_on_tiny_values(kind, heads, keys):
    """Value rows at the smallest scale, 2^-120: results are as small, lse is not moved."""
    b = Batch(kind, SINGLE, heads, quant=True, seed=40)
    requantise(b, lambda v, k: k.mul_(keys))
    want = b.run()[1].clone()
    requantise(b, lambda v, k: v.mul_(2.0 ** -119))
    assert float(b.pool.copy_scale.max()) == 2.0 ** -120
    b.check()
    assert float((b.lse - want).abs().max()) < 2.0 ** -15


@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
def test_the_sum_counts_tiny_values_beside_ordinary_ones(kind, heads):
    b = Batch(kind, SINGLE, heads, quant=True, seed=41)
    want = b.run()[1].clone()
    keep = torch.zeros(b.pool.copy.shape[1], dtype=torch.bool)
    for s in range(len(b.lens)):
        keep[b.slots(s)[::50]] = True
    size = torch.where(keep, 1.0, 2.0 ** -119).double().cuda()
    requantise(b, lambda v, k: v.mul_(size[:, None, None]))
    b.check()
    assert float((b.lse - want).abs().max()) < 2.0 ** -15
