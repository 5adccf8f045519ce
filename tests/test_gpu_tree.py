"""Attention of drafted trees over the paged cache against the 64-bit form."""
import math

import pytest
import torch

import position_independent_mla_gb300 as kv
from _keep import Tree
from _serve import Batch

pytestmark = pytest.mark.gpu

HEADS = {"mla": 16, "gqa": 32, "gqa4": 28, "mha": 32}


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind", sorted(HEADS))
def test_ragged_trees(kind, quant):
    Tree(kind, [(1, 1), (5, 130), (16, 577), (61, 61), (64, 391), (33, 129)], HEADS[kind],
         quant=quant).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads", [("mla", 128), ("mla", 3), ("gqa", 8), ("gqa", 64), ("gqa4", 4)])
def test_one_token_trees(kind, heads, quant):
    Tree(kind, [(1, 1), (1, 64), (1, 1000), (1, 129)], heads, quant=quant, seed=2).check()


@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", False), ("gqa4", True)])
def test_wide_trees_and_long_masks(kind, quant):
    # masks of several words, new tokens that cross key tiles at every offset
    Tree(kind, [(128, 300), (97, 131), (40, 168), (127, 127)], HEADS[kind], quant=quant, seed=3,
         extra_words=1).check()


@pytest.mark.parametrize("block", [1, 5, 16, 48, 128])
@pytest.mark.parametrize("kind,quant", [("mla", True), ("gqa", False)])
def test_block_sizes(kind, quant, block):
    Tree(kind, [(20, 300), (40, 259), (5, 5)], HEADS[kind], block=block, quant=quant, seed=4).check()


@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_strided(kind):
    Tree(kind, [(20, 300), (3, 90)], HEADS[kind], strided=True, seed=5).check()


@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_masks_of_any_kind(kind):
    # nothing at all, everything, later tokens, bits behind the last token, new tokens beyond the
    # cache (fewer keys than queries)
    n = 40
    masks = [[0] * n, [(1 << 64) - 1] * n, [1 << (n - 1 - i) for i in range(n)],
             [0xAAAAAAAAAA >> (i % 3) for i in range(n)]]
    t = Tree(kind, [(n, n), (n, 200), (n, 150), (n, 17)], HEADS[kind], masks=masks, seed=6)
    out, lse = t.check()
    assert torch.equal(out[:n], torch.zeros_like(out[:n]))
    assert bool((lse[:n] == -math.inf).all())


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_rows_that_a_query_does_not_see_may_hold_anything(kind, quant):
    t = Tree(kind, [(33, 200), (9, 9)], HEADS[kind], quant=quant, seed=7)
    slots = t.slots(0)
    bad = float("nan") if quant else float("inf")
    for j in (3, 17):  # some queries see these rows, others do not
        row = int(slots[200 - 33 + j])
        t.pool.copy[t.layer, row] = torch.full_like(t.pool.copy[t.layer, row].float(), bad).to(t.pool.copy.dtype)
    for s in range(2):  # rows behind the last key
        free = t.table[s].long() * t.block
        n = t.lens[s][1]
        k = torch.arange(n, -(-n // t.block) * t.block)
        rows = (free[k // t.block] + k % t.block).cuda()
        for part in (t.pool.copy, t.pool.rot):
            x = part[t.layer].view(torch.uint8 if part.element_size() == 1 else torch.int16)
            x[rows] = 0x7F if part.element_size() == 1 else 0x7FC0
    out, _ = t.run()
    want, _, tol, _ = t.reference()
    for i in range(33):
        sees = (t.masks[0][i] >> 3 | t.masks[0][i] >> 17) & 1
        assert bool(torch.isfinite(out[i].float()).all()) == (not sees), i
    ok = torch.isfinite(want)
    assert not ((out.double() - want).abs()[ok] > tol[ok]).any()


def test_a_chain_is_the_causal_chunk():
    lens = [(40, 700), (64, 64)]
    chain = [[(1 << i + 1) - 1 for i in range(n)] for n, _ in lens]
    t = Tree("gqa", lens, 32, masks=chain, seed=8)
    a = Batch("gqa", lens, 32, seed=8)
    for x, y in zip(t.check(), a.check()):
        assert (x.float() - y.float()).abs().max() < 0.05


def test_long_context_in_slices_and_equal_bits():
    t = Tree("gqa", [(60, 9000), (17, 300), (64, 5000)], 32, seed=9)
    first = [x.clone() for x in t.check()]
    for x, y in zip(first, t.run()):
        assert torch.equal(x, y)


def test_errors_of_the_device():
    t = Tree("gqa", [(8, 100), (8, 100)], 32, seed=10)
    t.attn.max_kv_len = 99
    t.ws = kv.tree_workspace(t.desc, t.attn, t.q)
    t.out.fill_(3.0)
    t.run(kv.KV_ERR_OUT_OF_RANGE)
    assert bool((t.out == 3.0).all())


def test_captured_and_replayed():
    t = Tree("mla", [(20, 300), (3, 90)], 16, seed=11)
    want, _ = t.check()
    want = want.clone()
    t.out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.kv_tree_attention(t.desc, t.layer, t.attn, t.mask, t.q, t.out, t.lse, t.ws)
    for _ in range(2):
        t.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t.out, want)


def test_tree_mask_of_parents():
    m = kv.tree_mask([[-1, 0, 0, 1], [-1] + list(range(39))], device="cpu")
    assert m.shape == (44, 2)
    assert m[:4, 0].tolist() == [1, 3, 5, 11] and m[:4, 1].tolist() == [0] * 4
    assert m[43].tolist() == [-1, 255]
