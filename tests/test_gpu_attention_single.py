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


def dominate(b, v, k, s, key, gap, others=None):
    """Key `key` of sequence s scores about `gap` (nats) with the first query head of every key
    head; `others`: what all keys of the sequence hold else (None: as they are)."""
    slots = b.slots(s).cuda()
    if others is not None:
        k[b.layer, slots] = others
    first = sum(n for n, _ in b.lens[:s])
    q = b.q[first, :: b.heads // b.h].double()
    k[b.layer, slots[key]] = q * (gap / b.scale / q.square().sum(-1, keepdim=True))


@pytest.mark.parametrize("gap", [3.0, 6.0, 11.0, 25.0])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -6, 2.0 ** -20])
@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64), ("mha", 32)])
def test_a_row_without_values_takes_no_precision_from_others(kind, heads, size, gap):
    """A value row of zeros (a null key, a blanked slot) is stored with scale 1; its weight adds
    nothing to the result, however large it is."""
    b = Batch(kind, [(1, 300), (1, 1000), (1, 129)], heads, quant=True, seed=42)

    def change(v, k):
        v.mul_(size)
        for s, key in enumerate((0, 700, 128)):
            dominate(b, v, k, s, key, gap)
            v[b.layer, b.slots(s)[key]] = 0.0
            v[b.layer, b.slots(s)[key], ::2, 5] = -0.0
    requantise(b, change).check()


def test_not_a_number_among_zeros_takes_no_precision_from_others():
    b = Batch("gqa", [(1, 1000)], 32, quant=True, seed=43)

    def change(v, k):
        v.mul_(2.0 ** -20)
        dominate(b, v, k, 0, 500, 11.0)
        v[b.layer, b.slots(0)[500]] = 0.0
        v[b.layer, b.slots(0)[500], :, 3] = float("nan")
    requantise(b, change).check()


@pytest.mark.parametrize("gap", [8.0, 13.0, 16.0])
@pytest.mark.parametrize("kind,heads,n", [("gqa", 32, 16000), ("gqa4", 64, 16000),
                                          ("mha", 32, 4000)])
def test_many_small_weights_beside_a_large_one(kind, heads, n, gap):
    """Thousands of equal keys far below one: each weight is small, not their sum."""
    b = Batch(kind, [(1, n), (1, 200)], heads, quant=True, seed=44)

    def change(v, k):
        v.abs_()
        dominate(b, v, k, 0, n // 3, gap, others=0.0)
    requantise(b, change).check()


@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
def test_values_of_far_apart_sizes(kind, heads):
    """Rows 2^-20 to 2^-12 of another's size, and a large row that is zero in half of its columns:
    there the small ones are all of the result.  A weight times its value's scale is held to
    2^-34 of the largest such product, a value is at most 448 scales."""
    b = Batch(kind, [(1, 700), (1, 3000)], heads, quant=True, seed=45)
    g = torch.Generator().manual_seed(5)
    size = torch.exp2(torch.randint(-20, -11, b.pool.copy.shape[1:2], generator=g).double()).cuda()

    def change(v, k):
        v.mul_(size[:, None, None])
        for s, key in enumerate((200, 1111)):
            dominate(b, v, k, s, key, 2.0)
            v[b.layer, b.slots(s)[key]] = 2.0
            v[b.layer, b.slots(s)[key], :, ::2] = 0.0
    requantise(b, change).check()


@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
def test_queries_with_a_channel_that_stands_out(kind, heads):
    """A query value 2^18 times the others, where the keys are zero: the others decide."""
    b = Batch(kind, [(1, 700), (1, 3000)], heads, quant=True, seed=46)

    def change(v, k):
        k[..., 0] = 0.0
    requantise(b, change)
    b.q[..., 0] = 2.0 ** 18
    b.q[::2, ..., 0] = -2.0 ** 18
    b.check()
