"""Attention over the paged cache against the 64-bit form: row shapes, pools,
lengths, masks, strides, and what a masked place may hold."""
import math

import pytest
import torch

import position_independent_mla_gb300 as kv
from _serve import Batch

pytestmark = pytest.mark.gpu

HEADS = {"mla": 16, "gqa": 32, "gqa4": 28, "mha": 32}
RAGGED = [(1, 1), (3, 130), (1, 577), (67, 67), (130, 391), (2, 64)]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind", sorted(HEADS))
def test_ragged_chunks(kind, quant):
    Batch(kind, RAGGED, HEADS[kind], quant=quant).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads", [("mla", 128), ("mla", 7), ("gqa", 8), ("gqa", 64),
                                        ("gqa4", 4), ("gqa4", 28), ("mha", 32)])
def test_single_tokens(kind, heads, quant):
    Batch(kind, [(1, 1), (1, 63), (1, 64), (1, 65), (1, 1000), (1, 128), (1, 129)], heads,
          quant=quant, seed=3).check()


@pytest.mark.parametrize("block", [1, 5, 16, 48, 128, 256])
@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", True), ("gqa4", False)])
def test_block_sizes(kind, quant, block):
    Batch(kind, [(1, 300), (40, 259), (5, 5)], HEADS[kind], block=block, quant=quant, seed=4).check()


@pytest.mark.parametrize("kind,quant", [("mla", False), ("mla", True), ("gqa", False),
                                        ("gqa", True)])
def test_lengths_around_tiles(kind, quant):
    lens = [(n, m) for n in (1, 31, 33, 128) for m in (127, 128, 129, 255, 257) if n <= m]
    Batch(kind, lens, HEADS[kind], quant=quant, seed=5).check()


@pytest.mark.parametrize("kind", ["mla", "gqa", "gqa4"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (100, 4), (130, 67), (5000, 4),
                                          (17, 1000)])
def test_window_and_sinks(kind, window, sinks):
    Batch(kind, [(1, 900), (70, 640), (33, 33), (1, 1), (300, 300), (1, 105)], HEADS[kind],
          window=window, sinks=sinks, seed=6).check()


def test_window_and_sinks_quantised():
    for kind in ("mla", "mha"):
        Batch(kind, [(1, 2000), (70, 640)], HEADS[kind], window=200, sinks=4, quant=True,
              seed=7).check()


@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_every_key_without_causal_mask(kind):
    Batch(kind, [(1, 200), (50, 333), (129, 64)], HEADS[kind], causal=False, seed=8).check()


@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_rows_that_see_nothing(kind):
    """More queries than cached tokens, an empty cache, sequences without queries."""
    b = Batch(kind, [(5, 3), (2, 0), (0, 40), (140, 6), (0, 0), (1, 0), (1, 2)], HEADS[kind], seed=9)
    out, lse = b.check()
    assert not out[5:7].float().any() and bool((lse[5:7] == -math.inf).all())


@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", False), ("gqa", True)])
def test_strided_queries_results_and_pools(kind, quant):
    b = Batch(kind, [(1, 70), (37, 200)], HEADS[kind], quant=quant, strided=True, seed=10)
    b.check()
    base = b.out.transpose(0, 1)
    wide = torch.as_strided(base, (b.heads, b.n, 24), base.stride(), base.storage_offset() + b.dv)
    assert bool((wide == 7.0).all()), "columns beside the result were written"


@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_peaked_and_huge_scores(kind):
    """Scores of thousands: the maximum carries the result, no overflow."""
    Batch(kind, [(1, 500), (64, 300)], HEADS[kind], q_scale=200.0, seed=11).check()


@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_long_context(kind):
    Batch(kind, [(1, 20011), (2, 9000)], HEADS[kind], seed=12).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads,lens", [("gqa", 32, [(1500, 5003)]), ("mla", 128, [(64, 5003)]),
                                             ("gqa", 32, [(1, 9001)] * 40),
                                             ("mla", 128, [(1, 6001)] * 40)])
def test_long_runs_of_whole_tiles_before_a_partial_one(kind, heads, lens, quant):
    """Every stage of the rings is reused many times within a block."""
    Batch(kind, lens, heads, quant=quant, seed=19).check()


@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", False), ("gqa4", True)])
def test_places_that_are_not_seen_may_hold_anything(kind, quant):
    """NaN beyond the cached tokens, in unused blocks, before the window."""
    b = Batch(kind, [(1, 333), (20, 200)], HEADS[kind], quant=quant, window=64, sinks=2, seed=13)
    keep = torch.zeros(b.pool.copy.shape[1], dtype=torch.bool)
    for s in range(len(b.lens)):
        seen = b.visible(s).any(0)
        keep[b.slots(s)[seen]] = True
    want, wl = (t.clone() for t in b.run())
    for t in (b.pool.copy, b.pool.rot):
        t[:, (~keep).cuda()] = torch.full((), math.nan, dtype=t.dtype, device="cuda")
    out, lse = b.run()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("part", ["copy", "rot"])
@pytest.mark.parametrize("kind", ["mla", "gqa"])
def test_a_later_tokens_row_does_not_reach_earlier_queries(kind, part, what):
    b = Batch(kind, [(150, 300), (9, 9)], HEADS[kind], seed=14)
    want, wl = (t.clone() for t in b.run())
    bad = b.slots(0)[220].cuda()  # seen by queries 70 and later of the first sequence
    getattr(b.pool, part)[b.layer, bad, 1::2] = what
    out, lse = b.run()
    assert torch.equal(out[:70], want[:70]) and torch.equal(out[150:], want[150:])
    assert torch.equal(lse[:70], wl[:70]) and torch.equal(lse[150:], wl[150:])
    # the odd value columns of the queries that see it cannot be finite; MLA's
    # values are part of its keys, so whole rows follow there
    assert not torch.isfinite(out[70:150, :, 1::2].float()).any()


def test_errors_on_the_device():
    b = Batch("gqa", [(3, 100), (2, 50)], 32, seed=15)
    want = b.run()[0].clone()
    b.table[0, 1] = 10 ** 6
    b.attn._tensors[2].copy_(b.table)
    b.run(kv.KV_ERR_OUT_OF_RANGE)
    assert torch.equal(b.out[3:], want[3:])
    b.attn.max_kv_len = 60  # the first sequence is longer than stated: skipped
    b.ws = kv.attn_workspace(b.desc, b.attn, b.q)
    b.out.fill_(7.0)
    b.run(kv.KV_ERR_OUT_OF_RANGE)
    assert bool((b.out[:3] == 7.0).all()) and torch.equal(b.out[3:], want[3:])


def test_other_stream_no_lse_and_used_workspace():
    b = Batch("mla", [(1, 700), (5, 90)], 128, seed=16)
    want = b.run()[0].clone()
    b.ws.fill_(255)
    b.out.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kv.kv_attention(b.desc, b.layer, b.attn, b.q, b.out, None, b.ws, stream=st)
    assert kv.kv_get_device_status(b.ws, st) == kv.KV_OK
    assert torch.equal(b.out, want)


@pytest.mark.parametrize("kind,heads", [("mla", 128), ("gqa", 32)])
def test_the_same_call_gives_the_same_bits(kind, heads):
    b = Batch(kind, [(1, 5000), (1, 77), (1, 3000)], heads, seed=17)
    a, al = (t.clone() for t in b.run())
    for _ in range(5):
        out, lse = b.run()
        assert torch.equal(out, a) and torch.equal(lse, al)


def test_offsets_beyond_32_bits():
    """A pool whose last rows lie more than 2^32 bytes after its base."""
    kind, slots = "mha", 64 * 8200  # 4.3 GB per part
    copy = torch.zeros(1, slots, 4096, dtype=torch.bfloat16, device="cuda")
    rot = torch.zeros(1, slots, 4096, dtype=torch.bfloat16, device="cuda")
    b = Batch(kind, [(1, 100), (3, 128)], 32, seed=18)
    want, wl = b.run()
    shift = 8200 - int(b.table.max()) - 1
    n = b.pool.copy.shape[1]
    copy[0, shift * 64:shift * 64 + n] = b.pool.copy[b.layer][: slots - shift * 64]
    rot[0, shift * 64:shift * 64 + n] = b.pool.rot[b.layer][: slots - shift * 64]
    table = (b.table + shift).cuda()
    desc = kv.pool_desc(copy, rot, 64, 32, 10000.0)
    attn = kv.attn_desc(b.attn._tensors[0], b.attn._tensors[1], table, 3, 128, b.scale)
    out, lse = torch.empty_like(b.out), torch.empty_like(b.lse)
    kv.kv_attention(desc, 0, attn, b.q, out, lse, kv.attn_workspace(desc, attn, b.q))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind,heads,lens", [("mla", 128, [(1, 700), (1, 300)]),
                                             ("gqa", 32, [(70, 700)]), ("gqa", 32, [(1, 700)]),
                                             ("gqa", 32, [(1, 9000)] * 3),
                                             ("mha", 32, [(40, 300)])])
@pytest.mark.parametrize("block", [0, 3])
def test_a_wait_that_runs_out_is_reported_and_ends(kind, heads, lens, block):
    """A block that gets no MMA gives up after the wait limit; the other blocks and
    the next call are not affected."""
    b = Batch(kind, lens, heads, seed=20)
    want, wl = (t.clone() for t in b.run())
    kv.kv_set_wait_limit_ns(20_000_000)
    kv.kv_set_attention_skip_block(block)
    try:
        b.run(kv.KV_ERR_TIMEOUT)
    finally:
        kv.kv_set_attention_skip_block(-1)
        kv.kv_set_wait_limit_ns(0)
    out, lse = b.run()
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_widened_rows_and_rows_beyond_that_workspace_agree():
    """Chunks over a quantised pool: widened first, or (max_kv_len stated so large that
    the widened rows would pass the limit) converted by every tile on its way."""
    for kind in ("gqa", "mla"):
        b = Batch(kind, [(40, 700), (33, 33)], HEADS[kind], quant=True, seed=21)
        out, lse = (t.clone() for t in b.check())
        assert kv.kv_last_launch_count() >= 2
        b.attn.max_kv_len = 1 << 20
        b.attn.max_blocks = b.table.shape[1]
        n = kv.kv_attention_workspace_size(b.desc, b.attn, b.n, b.heads)
        assert n < 1 << 30
        b.ws = kv.attn_workspace(b.desc, b.attn, b.q)
        b.check()


@pytest.mark.parametrize("kind,heads,quant", [("mla", 16, False), ("gqa", 32, True), ("gqa4", 28, False)])
@pytest.mark.parametrize("window", [130, 391, (1 << 31) - 1])
def test_windows_as_long_as_the_context(kind, heads, quant, window):
    """Also with more queries than keys, whose first positions are negative."""
    Batch(kind, [(150, 3), (1, 391), (130, 391)], heads, quant=quant, window=window, sinks=2,
          seed=22).check()


def test_workspaces_may_hold_anything_before_a_call():
    b = Batch("gqa", [(1, 700), (5, 130)], 32, seed=23)
    want = b.run()[0].clone()
    for byte in (0xFF, 0x01, 0x80):
        b.ws.fill_(byte)
        assert torch.equal(b.run()[0], want)
    kv.kv_set_wait_limit_ns(1_000_000)
    try:  # a call whose status is one word, after one with a word per block
        kv.kv_check_wait_timeout(b.ws, 1_000_000)
        assert kv.kv_get_device_status(b.ws) == kv.KV_ERR_TIMEOUT
    finally:
        kv.kv_set_wait_limit_ns(0)
    assert b.run()[0].equal(want)


def test_more_rows_than_32_bits_count_are_refused():
    b = Batch("gqa", [(1, 64)], 32, seed=24)
    a = kv.attn_desc(*b.attn._tensors, 1 << 29, 64, b.scale)
    assert kv.kv_attention_workspace_size(b.desc, a, 1 << 29, 32) == 0


@pytest.mark.parametrize("kind,heads,seqs,quant", [("mla", 16, 170, False), ("gqa4", 28, 170, True),
                                                   ("mha", 32, 90, False), ("gqa", 32, 170, False)])
def test_many_sequences(kind, heads, seqs, quant):
    """More sequences than slices are made for, and many units to an SM."""
    lens = [((7 * i) % 6, (7 * i) % 6 + (131 * i) % 640) for i in range(seqs)]
    Batch(kind, lens, heads, quant=quant, seed=25).check()


def test_a_long_sequence_among_short_ones():
    lens = [(1, 40 + i) for i in range(20)] + [(3, 20000)] + [(2, 9)] * 5
    for kind, heads in (("mla", 128), ("gqa", 32)):
        Batch(kind, lens, heads, seed=26).check()


def test_not_a_number_behind_the_last_token_of_single_queries():
    b = Batch("mla", [(1, 1000), (1, 65), (2, 700)], 128, seed=27)
    want, wl = (t.clone() for t in b.run())
    keep = torch.zeros(b.pool.copy.shape[1], dtype=torch.bool)
    for s in range(len(b.lens)):
        keep[b.slots(s)] = True
    for t in (b.pool.copy, b.pool.rot):
        t[:, (~keep).cuda()] = math.nan
    out, lse = b.run()
    assert torch.equal(out, want) and torch.equal(lse, wl)
