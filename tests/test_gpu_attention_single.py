"""Attention of one new token per sequence over head rows (the kernel of every
decode step with up to 16 query heads to a key head) against the 64-bit form."""
import math

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


# key heads, query heads: groups of 4, 7, 1, 9, 12 and 16
SHAPES_OF_ONE = [("gqa", 32), ("gqa4", 28), ("mha", 32), ("gqa", 72), ("gqa", 96), ("gqa4", 64)]
# a cluster joins the parts of these, a kernel of its own those of the others
SHORT = [(1, 577), (1, 1), (1, 127), (1, 128), (1, 129), (1, 900)]
LONG = [(1, 20011), (1, 9000), (1, 40), (1, 5003)] * 2


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("lens", [SHORT, LONG], ids=["short", "long"])
@pytest.mark.parametrize("kind,heads", SHAPES_OF_ONE)
def test_lengths_and_groups(kind, heads, lens, quant):
    Batch(kind, lens[:3] if kind == "mha" else lens, heads, quant=quant, seed=50).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (100, 4), (130, 67), (4096, 4),
                                          (17, 1000), (8191, 129)])
def test_window_and_sinks(kind, heads, window, sinks, quant):
    for lens in (SHORT, [(1, 20011), (1, 105), (1, 9000)]):
        Batch(kind, lens, heads, window=window, sinks=sinks, quant=quant, seed=51).check()


@pytest.mark.parametrize("quant", [False, True])
def test_window_and_sinks_of_a_key_head_to_a_query_head(quant):
    Batch("mha", [(1, 9000), (1, 105)], 32, window=4096, sinks=4, quant=quant, seed=51).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("block", [1, 5, 8, 16, 24, 32, 48, 128, 256, 384])
@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
def test_block_sizes(kind, heads, block, quant):
    Batch(kind, [(1, 300), (1, 1000), (1, 5)], heads, block=block, quant=quant, seed=52).check()
    Batch(kind, [(1, 4000), (1, 77)], heads, block=block, quant=quant, window=1000, sinks=70,
          seed=53).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("block", [16, 48, 64, 256])
@pytest.mark.parametrize("window", [0, 200])
def test_places_that_are_not_seen_may_hold_anything(window, block, quant):
    """NaN values, keys and scales beyond the cached tokens, in unused blocks, before the window."""
    for kind, heads, lens in (("gqa", 32, SHORT), ("gqa4", 64, [(1, 3000), (1, 260)])):
        b = Batch(kind, lens, heads, block=block, quant=quant, window=window,
                  sinks=3 if window else 0, seed=54)
        keep = torch.zeros(b.pool.copy.shape[1], dtype=torch.bool)
        for s in range(len(b.lens)):
            keep[b.slots(s)[b.visible(s).any(0)]] = True
        want, wl = (t.clone() for t in b.run())
        for t in (b.pool.copy, b.pool.rot, b.pool.copy_scale, b.pool.rot_scale):
            if t is not None:
                t[:, (~keep).cuda()] = torch.full((), math.nan, dtype=t.dtype, device="cuda")
        out, lse = b.run()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("quant", [False, True])
def test_a_seen_value_that_is_not_a_number_stays_in_its_column(quant):
    b = Batch("gqa", [(1, 700), (1, 300)], 32, quant=quant, seed=55)
    want, wl = (t.clone() for t in b.run())
    at = b.slots(0)[400].cuda()
    b.pool.copy[b.layer, at, 5] = torch.full((), math.nan, dtype=b.pool.copy.dtype, device="cuda")
    out, lse = b.check()
    assert torch.equal(lse, wl) and torch.equal(out[1], want[1])
    assert torch.equal(out[0, 4:], want[0, 4:])


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
def test_strided_queries_results_and_pools(kind, heads, quant):
    for lens in ([(1, 70), (1, 700)], [(1, 9000), (1, 3)] * 4):
        b = Batch(kind, lens, heads, quant=quant, strided=True, seed=56)
        b.check()
        base = b.out.transpose(0, 1)
        wide = torch.as_strided(base, (b.heads, b.n, 24), base.stride(),
                                base.storage_offset() + b.dv)
        assert bool((wide == 7.0).all()), "columns beside the result were written"


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("q_scale", [1e-6, 200.0])
def test_peaked_flat_and_huge_scores(q_scale, quant):
    for kind, heads in (("gqa", 32), ("gqa4", 64)):
        Batch(kind, [(1, 500), (1, 2000)], heads, q_scale=q_scale, quant=quant, seed=57).check()


@pytest.mark.parametrize("quant", [False, True])
def test_empty_caches_sequences_without_queries_no_causal_mask(quant):
    lens = [(1, 0), (0, 40), (1, 300), (0, 0), (1, 2)]
    for causal in (True, False):
        out, lse = Batch("gqa", lens, 32, quant=quant, causal=causal, seed=58).check()
        assert not out[0].float().any() and bool((lse[0] == -math.inf).all())
    Batch("gqa", [(1, 0), (1, 0)], 32, quant=quant, seed=59).check()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("long", [200, 9000])
def test_errors_on_the_device(long, quant):
    b = Batch("gqa", [(1, long), (1, 150)], 32, quant=quant, seed=60)
    want, wl = (t.clone() for t in b.run())
    for bad in (10 ** 6, -1):
        b.attn._tensors[2].copy_(b.table)
        b.attn._tensors[2][0, 1] = bad
        b.run(kv.KV_ERR_OUT_OF_RANGE)
        assert torch.equal(b.out[1], want[1]) and torch.equal(b.lse[1], wl[1])
        assert torch.isfinite(b.out.float()).all()
    b.attn._tensors[2].copy_(b.table)
    for name, value in (("max_kv_len", 160), ("max_blocks", None)):
        b.out.fill_(7.0)
        if value:
            b.attn.max_kv_len = value  # the first sequence is longer than stated: skipped
            b.ws = kv.attn_workspace(b.desc, b.attn, b.q)
        else:                          # longer than its row of the table
            b.attn.max_kv_len = long
            t = b.attn._tensors[2][:, :3].contiguous()
            b.attn.d_block_tables, b.attn.max_blocks = t.data_ptr(), 3
            b.ws = kv.attn_workspace(b.desc, b.attn, b.q)
        b.run(kv.KV_ERR_OUT_OF_RANGE)
        assert bool((b.out[0] == 7.0).all()), name
        # the keys may be cut elsewhere: as near to the 64-bit form as any call
        want, _, bound, _ = b.reference()
        assert bool(((b.out[1].double() - want[1]).abs() <= bound[1]).all()), name


@pytest.mark.parametrize("quant", [False, True])
def test_two_new_tokens_where_one_was_stated(quant):
    b = Batch("gqa", [(1, 100), (1, 70), (1, 300)], 32, quant=quant, seed=61)
    want = b.run()[0].clone()
    b.attn._tensors[0].copy_(torch.tensor([0, 0, 2, 3], dtype=torch.int32))
    b.out.fill_(7.0)
    b.run(kv.KV_ERR_OUT_OF_RANGE)
    assert bool((b.out[:2] == 7.0).all()) and torch.equal(b.out[2], want[2])


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("heads,lens", [(32, SHORT), (64, LONG)])
def test_equal_calls_any_workspace_other_stream_no_lse(heads, lens, quant):
    b = Batch("gqa4", lens, heads, quant=quant, seed=62)
    want, wl = (t.clone() for t in b.run())
    for byte in (0, 0xFF, 0x7F):
        b.ws.fill_(byte)
        out, lse = b.run()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    b.out.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kv.kv_attention(b.desc, b.layer, b.attn, b.q, b.out, None, b.ws, stream=st)
    assert kv.kv_get_device_status(b.ws, st) == kv.KV_OK
    assert torch.equal(b.out, want)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads", [("gqa", 32), ("gqa4", 64)])
@pytest.mark.parametrize("lens", [SHORT, LONG], ids=["short", "long"])
def test_a_wait_that_runs_out_is_reported_and_ends(lens, kind, heads, quant):
    b = Batch(kind, lens, heads, quant=quant, seed=63)
    want, wl = (t.clone() for t in b.run())
    for block in (0, 4):  # with keys in every batch
        kv.kv_set_wait_limit_ns(20_000_000)
        kv.kv_set_attention_skip_block(block)
        try:
            b.run(kv.KV_ERR_TIMEOUT)
        finally:
            kv.kv_set_attention_skip_block(-1)
            kv.kv_set_wait_limit_ns(0)
        out, lse = b.run()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("quant", [False, True])
def test_offsets_beyond_32_bits(quant):
    """A pool whose last rows lie more than 2^32 bytes after its base."""
    blocks = 17000 if quant else 8300  # of 64 rows of 4096 bytes or twice that
    b = Batch("mha", [(1, 100), (1, 700)], 32, quant=quant, seed=64)
    want, wl = (t.clone() for t in b.run())
    n, shift = b.pool.copy.shape[1], blocks - b.pool.copy.shape[1] // 64
    parts = []
    for name in ("copy", "rot", "copy_scale", "rot_scale"):
        t = getattr(b.pool, name)
        if t is None:
            parts.append(None)
            continue
        big = torch.zeros(1, blocks * 64, t.shape[2], dtype=t.dtype, device="cuda")
        big[0, shift * 64:shift * 64 + n] = t[b.layer]
        parts.append(big)
    copy, rot, cs, rs = parts
    assert copy.nbytes > 1 << 32
    desc = (kv.quant_pool_desc(copy, cs, rot, rs, 64, 32) if quant
            else kv.pool_desc(copy, rot, 64, 32, 10000.0))
    table = (b.table + shift).cuda()
    attn = kv.attn_desc(b.attn._tensors[0], b.attn._tensors[1], table, 1, 700, b.scale)
    out, lse = torch.empty_like(b.out), torch.empty_like(b.lse)
    kv.kv_attention(desc, 0, attn, b.q, out, lse, kv.attn_workspace(desc, attn, b.q))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind,heads", [("gqa", 72), ("gqa", 128), ("gqa4", 68), ("gqa4", 200),
                                        ("gqa4", 512), ("mla", 9), ("mla", 100)])
def test_large_groups_beside_it(kind, heads, quant):
    """Chunks, and single tokens of more than 16 query heads to a key head: the other kernels."""
    Batch(kind, [(1, 300), (1, 1), (1, 2000)], heads, quant=quant, seed=65).check()
    Batch(kind, [(3, 300), (30, 700), (1, 129)], heads, quant=quant, seed=66).check()
    Batch(kind, [(2, 300), (40, 700)], heads, quant=quant, window=100, sinks=3, seed=67).check()
