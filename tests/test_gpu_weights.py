"""What each cached key receives of the queries' attention, against the 64-bit form."""
import math

import pytest
import torch

import position_independent_mla_gb300 as kv
from _keep import Sums

pytestmark = pytest.mark.gpu

HEADS = {"mla": 16, "gqa": 32, "gqa4": 28, "mha": 32}


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind", sorted(HEADS))
def test_ragged_chunks(kind, quant):
    Sums(kind, [(1, 1), (3, 130), (1, 577), (67, 67), (130, 391), (2, 64)], HEADS[kind],
         quant=quant).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads", [("mla", 128), ("mla", 7), ("gqa", 8), ("gqa", 64),
                                        ("gqa4", 4), ("gqa4", 28), ("mha", 32)])
def test_single_tokens(kind, heads, quant):
    Sums(kind, [(1, 1), (1, 63), (1, 64), (1, 65), (1, 1000), (1, 128), (1, 129)], heads,
         quant=quant, seed=3).check()


@pytest.mark.parametrize("keep", [0.0, 0.95, 1.0, 2.5])
def test_keep(keep):
    s = Sums("gqa", [(1, 300), (9, 140)], 32, keep=keep, seed=2)
    if keep == 0.0:
        s.weights[:, ::7] = float("nan")  # is not read
        old = s.weights.clone()
        got = s.run()
        assert not bool(torch.isnan(got[0, :300]).any() or torch.isnan(got[1, :140]).any())
        s.weights = torch.nan_to_num(old, nan=0.5)
    s.check()


@pytest.mark.parametrize("block", [1, 5, 16, 48, 128, 256])
@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", True), ("gqa4", False), ("mla", True)])
def test_block_sizes(kind, quant, block):
    Sums(kind, [(1, 300), (40, 259), (5, 5)], HEADS[kind], block=block, quant=quant, seed=4).check()


@pytest.mark.parametrize("kind", ["mla", "gqa", "gqa4"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (100, 4), (130, 67), (5000, 4),
                                          (17, 1000)])
def test_window_and_sinks(kind, window, sinks):
    Sums(kind, [(1, 900), (70, 640), (33, 33), (1, 1), (300, 300), (1, 105)], HEADS[kind],
         window=window, sinks=sinks, seed=6).check()


@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_every_key_without_causal_mask(kind):
    Sums(kind, [(1, 200), (50, 333), (129, 64)], HEADS[kind], causal=False, seed=8).check()


@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", False), ("gqa", True), ("mha", False)])
def test_strided_and_heads_outside_tokens(kind, quant):
    Sums(kind, [(20, 300), (3, 90)], HEADS[kind], strided=True, quant=quant, seed=5).check()


def test_empty_sequences():
    # no queries: older steps fade all the same; no keys: nothing to write; more queries than keys
    s = Sums("gqa", [(0, 200), (3, 0), (9, 5), (2, 130)], 32, keep=0.5, seed=9)
    old = s.weights.clone()
    s.check()
    assert torch.equal(s.weights[0, :200], old[0, :200] * 0.5)
    assert torch.equal(s.weights[1], old[1])


@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", False), ("gqa", True)])
def test_a_key_that_is_nan_has_no_part_in_others(kind, quant):
    s = Sums(kind, [(5, 200), (70, 150)], HEADS[kind], quant=quant, seed=10)
    rows = torch.stack([s.slots(0)[7], s.slots(1)[149]]).cuda()
    x = s.pool.rot[s.layer].view(torch.uint8 if s.pool.rot.element_size() == 1 else torch.int16)
    x[rows, 3] = 0x7F if s.pool.rot.element_size() == 1 else 0x7FC0
    # rows behind the last key of a block
    for q in range(2):
        m = s.lens[q][1]
        last = int(s.table[q][m // s.block]) * s.block + m % s.block
        x[last:last + 3] = 0x7F if s.pool.rot.element_size() == 1 else 0x7FC0
    old, got = s.weights.clone(), s.run()
    # (its last key: seen by the last query alone)
    for q, k in ((0, 7), (1, 149)):
        assert math.isnan(float(got[q, k]))
        got[q, k] = old[q, k]
        assert bool(torch.isfinite(got[q]).all())


def test_queries_that_count_nothing():
    s = Sums("gqa", [(4, 200)], 32, seed=11)
    s.lse[1] = -math.inf
    s.lse[2, 5:9] = -math.inf
    s.check()


def test_queries_of_another_sequence_have_no_part():
    s = Sums("gqa", [(5, 300), (3, 290)], 32, seed=12)
    s.q[5:] = float("nan")
    s.lse[5:] = float("nan")
    old = s.weights.clone()
    got = s.run()
    assert bool(torch.isfinite(got[0]).all())
    assert bool(torch.isnan(got[1, :287]).all()) and torch.equal(got[1, 290:], old[1, 290:])


def test_many_queries_over_a_long_context_and_equal_bits():
    s = Sums("gqa", [(700, 3000), (64, 513)], 32, keep=0.0, seed=13)
    first = s.check().clone()
    assert torch.equal(first[0, :3000], s.run().double()[0, :3000])


def test_scores_far_apart():
    Sums("gqa", [(9, 400)], 32, q_scale=12.0, seed=14).check()


def test_sums_to_the_number_of_rows():
    s = Sums("gqa4", [(33, 700)], 28, keep=0.0, seed=15)
    assert abs(float(s.run()[0, :700].double().sum()) - 33 * 28) < 1e-3 * 33 * 28


def test_errors_of_the_device():
    s = Sums("gqa", [(3, 200), (3, 100)], 32, seed=16)
    s.table_dev = s.attn._tensors[2]
    s.table_dev[0, 1] = 10 ** 6
    old, got = s.weights.clone(), s.run(kv.KV_ERR_OUT_OF_RANGE)
    assert torch.equal(got[0, 64:128], old[0, 64:128])  # nothing is added to the keys of that block
    assert bool((got[0, :64] > old[0, :64]).all())
    s.attn.max_kv_len = 150
    s.wws = kv.weights_workspace(s.desc, s.attn, s.q)
    old, got = s.weights.clone(), s.run(kv.KV_ERR_OUT_OF_RANGE)
    assert torch.equal(got[0], old[0]) and bool((got[1, :90] > old[1, :90]).all())


def test_a_wait_that_runs_out():
    s = Sums("gqa", [(3, 200)], 32, seed=17)
    old = s.weights.clone()
    kv.kv_set_wait_limit_ns(2_000_000)
    kv.kv_set_attention_skip_block(1)
    try:
        s.run(kv.KV_ERR_TIMEOUT)
        # the other key tile, of the blocks that went on
        n = 128 if bool(torch.equal(s.weights[0, :128], old[0, :128])) else 0
        assert torch.equal(s.weights[0, 200:], old[0, 200:])
        assert n == 128
    finally:
        kv.kv_set_attention_skip_block(-1)
        kv.kv_set_wait_limit_ns(0)
    s.weights.copy_(old)
    s.check()


@pytest.mark.parametrize("kind,heads,lens,quant", [
    ("mla", 16, [(20, 300), (3, 90)], False), ("mla", 16, [(2, 300), (3, 90)], True),
    ("gqa", 32, [(1, 300), (1, 90)], False), ("gqa", 32, [(90, 300), (40, 500)], False)])
def test_captured_and_replayed(kind, heads, lens, quant):
    s = Sums(kind, lens, heads, keep=0.0, seed=18, quant=quant)
    want = s.check().clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.kv_attention_weights(s.desc, s.layer, s.attn, s.q, s.lse, s.weights, 0.0, s.wws)
    for _ in range(2):
        s.weights.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        for q, (_, m) in enumerate(s.lens):
            assert torch.equal(s.weights[q, :m].double(), want[q, :m])


@pytest.mark.parametrize("kind,quant", [("mla", False), ("mla", True), ("gqa", False), ("gqa", True)])
def test_no_queries_at_all(kind, quant):
    s = Sums(kind, [(0, 200), (0, 3), (0, 0)], HEADS[kind], keep=0.25, quant=quant, seed=27)
    old = s.weights.clone()
    s.run()
    for q, m in enumerate((200, 3, 0)):
        assert torch.equal(s.weights[q, :m], old[q, :m] * 0.25)
        assert torch.equal(s.weights[q, m:], old[q, m:])


def test_on_another_stream():
    s = Sums("gqa", [(3, 500)], 32, seed=28)
    old = s.weights.clone()
    want = s.run().clone()
    s.weights.copy_(old)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        kv.kv_attention_weights(s.desc, s.layer, s.attn, s.q, s.lse, s.weights, s.keep, s.wws)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(s.weights, want)


@pytest.mark.parametrize("quant", [False, True])
def test_many_queries_a_wait_that_runs_out(quant):
    s = Sums("gqa", [(300, 1000), (40, 513)], 32, seed=19, quant=quant)
    old = s.weights.clone()
    kv.kv_set_wait_limit_ns(2_000_000)
    kv.kv_set_attention_skip_block(3)
    try:
        s.run(kv.KV_ERR_TIMEOUT)
    finally:
        kv.kv_set_attention_skip_block(-1)
        kv.kv_set_wait_limit_ns(0)
    assert torch.equal(s.weights, old)  # what parts of a key's sum there are is not stored
    s.check()


@pytest.mark.parametrize("kind,heads,quant", [("gqa", 8, False), ("gqa", 40, False), ("gqa4", 28, True),
                                              ("mha", 32, False), ("gqa4", 12, False), ("gqa", 64, True)])
def test_many_queries_of_several_sequences(kind, heads, quant):
    lens = [(260, 1000), (1, 300), (0, 40), (129, 129), (400, 2000), (17, 700)]
    Sums(kind, lens, heads, quant=quant, seed=20, keep=0.5).check()


def test_many_queries_with_more_units_than_parts():
    lens = [(70 + i, 200 + 90 * i) for i in range(40)]
    Sums("gqa4", lens, 28, seed=21).check()


@pytest.mark.parametrize("window,sinks", [(300, 4), (40, 300), (1, 0)])
def test_many_queries_under_a_window(window, sinks):
    Sums("gqa", [(500, 1500), (200, 200)], 32, window=window, sinks=sinks, seed=22).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads,n", [("gqa", 8, 1), ("gqa", 16, 1), ("gqa", 24, 1), ("gqa", 32, 4),
                                          ("gqa", 64, 2), ("gqa", 128, 1), ("gqa4", 4, 3), ("gqa4", 28, 2),
                                          ("mha", 32, 1), ("mha", 32, 3), ("mha", 32, 5), ("mha", 32, 16),
                                          ("mla", 5, 2), ("mla", 16, 3), ("mla", 48, 1), ("mla", 128, 1)])
def test_few_rows(kind, heads, n, quant):
    Sums(kind, [(n, 130), (1, 300), (n, 2000), (0, 65), (n, n)], heads, quant=quant, seed=23,
         keep=0.7).check()


@pytest.mark.parametrize("kind,heads,quant", [("gqa", 32, False), ("gqa", 32, True), ("mla", 64, False)])
def test_few_rows_in_runs(kind, heads, quant):
    # so many sequences that a block takes several key tiles
    lens = [(1, 900 + 17 * i) for i in range(48)]
    Sums(kind, lens, heads, quant=quant, seed=24, block=16).check()


@pytest.mark.parametrize("kind,heads,quant", [("gqa", 32, False), ("gqa", 32, True), ("mla", 64, False)])
def test_few_rows_under_a_window(kind, heads, quant):
    lens = [(1, 1100 + 37 * i) for i in range(40)]
    Sums(kind, lens, heads, quant=quant, seed=25, window=200, sinks=4).check()


def test_few_rows_queries_far_apart_over_quantised_rows():
    s = Sums("gqa", [(2, 700)], 32, quant=True, seed=26)
    s.q[0, :, ::3] *= 2.0 ** -12
    s.q[1, 5] = 0.0
    s.lse = s.scores_lse().float().contiguous()
    s.check()


@pytest.mark.parametrize("kind,heads,lens", [
    ("gqa", 32, [(1, 300), (2, 100)]), ("gqa", 32, [(20, 300), (3, 100)]),
    ("gqa", 32, [(90, 300), (300, 700)]), ("mla", 16, [(2, 300), (1, 100)]), ("mla", 16, [(40, 300)])])
def test_heads_that_share_their_queries(kind, heads, lens):
    s = Sums(kind, lens, heads, seed=29)
    s.q = s.q[:, :1].expand(-1, heads, -1)  # no stride between heads: rows that boxes do not fit
    assert s.q.stride(1) == 0
    s.lse = s.scores_lse().float().contiguous()
    s.check()


@pytest.mark.parametrize("heads,quant", [(8 * 80, False), (8 * 100, True), (8 * 128, False)])
def test_many_heads_to_a_key_head(heads, quant):
    Sums("gqa", [(3, 300), (1, 140)], heads, seed=30, quant=quant).check()
    Sums("gqa", [(1, 300), (1, 140)], heads, seed=31, quant=quant).check()
