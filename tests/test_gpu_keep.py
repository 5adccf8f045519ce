"""The choice of the tokens that stay, the move of their rows, and the operators of a bounded
cache and of drafted tokens one after another."""
import math

import numpy as np
import pytest
import torch

import position_independent_mla_gb300 as kv
import synth
from _gpu import bf16_to_f64, ordered
from _keep import ref_select
from _serve import SHAPES, bf16_rows, empty_quant

pytestmark = pytest.mark.gpu


def select(weights, lens, budget, sinks, recent, most=None, kept=True, status=kv.KV_OK):
    n = len(lens)
    most = most if most is not None else max(1, max(min(a, b) for a, b in zip(lens, budget)))
    keep = torch.full((n, most + 3), -7, dtype=torch.int32, device="cuda")[:, :most]
    count = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    kw = torch.full((n, most), -5.0, device="cuda") if kept else None
    ws = kv.evict_workspace(n, weights.shape[1])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv.kv_evict_select(weights, i32(lens), i32(budget), sinks, recent, keep, count, kw, ws)
    assert kv.kv_get_device_status(ws) == status
    return keep, count, kw


def check_select(weights, lens, budget, sinks, recent):
    keep, count, kw = select(weights.cuda(), lens, budget, sinks, recent)
    for s, want in enumerate(ref_select(weights, lens, budget, sinks, recent)):
        assert int(count[s]) == len(want)
        assert keep[s, : len(want)].tolist() == want
        assert bool((keep[s, len(want):] == -7).all()) and bool((kw[s, len(want):] == -5.0).all())
        got, exp = kw[s, : len(want)].cpu(), weights[s, want]
        assert torch.equal(got.view(torch.int32), exp.view(torch.int32))


def heavy(seed, n, m):
    g = torch.Generator().manual_seed(seed)
    x = torch.exp(2 * torch.randn(n, m, generator=g))
    x[torch.rand(n, m, generator=g) < 0.1] = 0.0
    return x


@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 64), (1, 0), (0, 31), (700, 700)])
def test_select_ragged(sinks, recent):
    lens = [1, 2, 31, 32, 33, 577, 1000, 1024, 1025, 0]
    check_select(heavy(1, 10, 1100), lens, [1, 1, 7, 32, 20, 300, 1, 999, 600, 5], sinks, recent)


@pytest.mark.parametrize("seqs,m", [(1, 4096), (1, 5000), (2, 16384), (1, 70001), (80, 300), (3, 33000)])
def test_select_in_clusters(seqs, m):
    lens = [m - 3 * i for i in range(seqs)]
    check_select(heavy(2, seqs, m + 5), lens, [max(1, n // 3) for n in lens], 4, 9)


def test_select_beyond_what_a_block_holds():
    check_select(heavy(3, 80, 60000), [60000 - i for i in range(80)], [100 + 500 * i for i in range(80)], 4, 50)


def test_select_ties_and_odd_values():
    w = torch.ones(6, 3000)
    w[1, ::3] = 0.0
    w[1, 1::3] = -0.0
    w[2, 100:200] = float("nan")
    w[3] = float("nan")
    w[4, ::5], w[4, 1::5], w[4, 2::5] = math.inf, -math.inf, -1.5
    w[5] = torch.arange(3000) % 7
    for b in (1, 500, 1500, 2999, 3000):
        check_select(w, [3000] * 6, [b] * 6, 0, 0)
        check_select(w, [2900] * 6, [b] * 6, 3, 40)


def test_select_budgets_of_the_fixed_tokens():
    w = heavy(5, 1, 200)
    for b in range(0, 40):
        check_select(w, [150], [b], 10, 20)


def test_select_equal_keys_in_one_bin():
    # weights whose first digits agree: found by the last ones
    bits = torch.full((2, 5000), 0x3F800000, dtype=torch.int32)
    bits[0] += torch.arange(5000) % 900
    bits[1] += (torch.arange(5000) * 7919) % 5000
    check_select(bits.view(torch.float32), [5000, 4999], [2500, 77], 2, 2)


def test_select_refuses_on_the_device():
    w = heavy(6, 4, 100).cuda()
    keep, count, _ = select(w, [101, -1, 100, 50], [5, 5, 60, 60], 0, 0, most=50,
                            status=kv.KV_ERR_OUT_OF_RANGE)
    assert count.tolist() == [-1, -1, -1, 50]
    assert bool((keep[:3] == -7).all()) and keep[3].tolist() == list(range(50))
    _, count, _ = select(w, [100, 100, 100, 50], [-1, 5, 5, 5], 0, 0, kept=False,
                         status=kv.KV_ERR_OUT_OF_RANGE, most=5)
    assert count.tolist() == [-1, 5, 5, 5]


# ---------------------------------------------------------------------------

class Pool:
    """A paged pool and its parts as the reference moves them."""

    def __init__(self, kind, lens, layers=2, block=64, quant=False, pair=0, spare=0, seed=1, pad=0):
        g = torch.Generator().manual_seed(seed)
        cd, self.h, self.d, self.base = SHAPES[kind]
        self.kind, self.block, self.pair, self.quant, self.layers = kind, block, pair, quant, layers
        per = max(1, -(-(max(lens) + spare) // block))
        blocks = len(lens) * per + 2
        self.table = torch.randperm(blocks, generator=g)[: len(lens) * per].int().view(len(lens), per)
        slots = blocks * block
        copy, rot = bf16_rows(g, layers, slots, cd), bf16_rows(g, layers, slots, self.h * self.d)
        if quant:
            self.p = empty_quant(kind, layers, slots, block, pad=pad)
            src = kv.pool_desc(copy.cuda(), rot.cuda(), 1, self.h, self.base)
            ws = kv.quant_workspace(self.p.desc)
            kv.kv_quantize(src, None, self.p.desc, 0, slots,
                           torch.arange(slots, dtype=torch.int32, device="cuda"), ws)
            self.desc = self.p.desc
            self.parts = {k: getattr(self.p, k) for k in ("copy", "copy_scale", "rot", "rot_scale")
                          if getattr(self.p, k) is not None}
        else:
            wide = torch.zeros(layers, slots, cd + self.h * self.d + 8 * pad, dtype=torch.bfloat16,
                               device="cuda")
            wide[..., :cd], wide[..., cd:cd + self.h * self.d] = copy.cuda(), rot.cuda()
            self.parts = {"copy": wide[..., :cd], "rot": wide[..., cd:cd + self.h * self.d]}
            self.desc = kv.pool_desc(self.parts["copy"], self.parts["rot"], block, self.h, self.base, pair)

    def bits(self):
        torch.cuda.synchronize()
        views = {1: torch.uint8, 2: torch.int16, 4: torch.int32}
        return {k: v.view(views[v.element_size()]).cpu().numpy().copy() for k, v in self.parts.items()}

    def slot(self, s, p):
        return self.table[s].numpy().astype(np.int64)[p // self.block] * self.block + p % self.block

    def turn(self, bits, m):
        """R(-m) of bf16 rows [L, N, h*d] (bits) in 64 bits, rounded to bf16's bits."""
        x = bf16_to_f64(bits.view(np.uint16)).reshape(*bits.shape[:2], self.h, self.d)
        j = np.arange(self.d // 2)
        a = -m[:, None].astype(np.float64) * self.base ** (-2.0 * j / self.d)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        y = np.empty_like(x)
        if self.pair:
            u, v = x[..., 0::2], x[..., 1::2]
            y[..., 0::2], y[..., 1::2] = u * c - v * s, u * s + v * c
        else:
            u, v = x[..., : self.d // 2], x[..., self.d // 2:]
            y[..., : self.d // 2], y[..., self.d // 2:] = u * c - v * s, u * s + v * c
        return torch.from_numpy(y.reshape(bits.shape)).to(torch.bfloat16).view(torch.int16).numpy()

    def check(self, keep, first=None, rotate=True, status=kv.KV_OK, run=None):
        """Moves the rows of ``keep`` (lists) and compares: bit for bit where nothing turns, within
        one step of bf16 where the fp64 value may lie on either side of a border."""
        want = self.bits()
        n = len(keep)
        most = max(1, max(len(k) for k in keep))
        lists = torch.full((n, most + 2), 12345678, dtype=torch.int32)
        for s, k in enumerate(keep):
            k = np.array(k, dtype=np.int64)
            lists[s, : len(k)] = torch.from_numpy(k).int()
            b = 0 if first is None else first[s]
            i = np.arange(len(k))
            go = k != i
            src, dst, m = self.slot(s, b + k[go]), self.slot(s, b + i[go]), (k - i)[go]
            for name, t in want.items():
                rows = t[:, src]
                if name == "rot" and rotate:
                    rows = self.turn(rows, m)
                t[:, dst] = rows
        lists, table = lists.cuda(), self.table.cuda()
        keep_t = lists[:, :most]
        count = torch.tensor([len(k) for k in keep], dtype=torch.int32, device="cuda")
        first_t = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
        ws = kv.compact_workspace(self.desc, n, table.shape[1], most)
        more = dict(rope_base=self.base, pair_convention=self.pair) if self.quant and rotate else {}
        kv.kv_compact(self.desc, table, first_t, keep_t, count, rotate, ws, **more)
        assert kv.kv_get_device_status(ws) == status
        got = self.bits()
        for name in want:
            if name == "rot" and rotate:
                far = np.abs(ordered(got[name].view(np.uint16)) - ordered(want[name].view(np.uint16)))
                tiny = np.abs(bf16_to_f64(got[name].view(np.uint16)) - bf16_to_f64(want[name].view(np.uint16))) < 1e-6
                assert bool(((far <= 1) | tiny).all()), (name, int((far > 1).sum()))
                # rounded once: but for values on a border, all are equal
                assert (far > 0).mean() < 1e-4
            else:
                assert np.array_equal(got[name], want[name]), name


def subset(seed, n, c):
    return sorted(np.random.RandomState(seed).permutation(n)[:c].tolist())


KINDS = [("mla", False, 0), ("mla", False, 1), ("mla", True, 0), ("mla", True, 1), ("gqa", False, 0),
         ("gqa", False, 1), ("gqa4", False, 0), ("mha", False, 0)]


@pytest.mark.parametrize("kind,quant,pair", KINDS)
def test_compact_turned(kind, quant, pair):
    lens = [500, 65, 300, 1, 64, 200]
    keep = [subset(1, 500, 250), list(range(65)), subset(2, 300, 299), [0], [63], []]
    Pool(kind, lens, quant=quant, pair=pair, layers=3).check(keep)


@pytest.mark.parametrize("kind,quant", [("mla", False), ("mla", True), ("gqa", False), ("gqa", True),
                                        ("gqa4", False), ("gqa4", True), ("mha", False), ("mha", True)])
def test_compact_as_they_are(kind, quant):
    lens = [400, 130, 300]
    keep = [subset(3, 400, 77), subset(4, 130, 100), list(range(299, 300))]
    Pool(kind, lens, quant=quant, pad=1).check(keep, rotate=False)


@pytest.mark.parametrize("block", [1, 7, 16, 64, 100])
def test_compact_block_sizes(block):
    Pool("mla", [300, 90], block=block).check([subset(5, 300, 150), subset(6, 90, 50)])


def test_compact_one_gap_and_dense_lists():
    # every row waits for the tile before its own; then whole tiles that no row leaves
    n = 2000
    Pool("mla", [n], layers=5).check([list(range(1, n))])
    Pool("gqa", [n], layers=2).check([list(range(700)) + list(range(703, n))])
    Pool("mla", [n], layers=2).check([list(range(0, n, 2))])


def test_compact_many_layers_and_sequences():
    lens = [257] * 40
    Pool("mla", lens, layers=61).check([subset(i, 257, 100 + i) for i in range(40)], rotate=False)


def test_compact_far_positions():
    n = 40000
    Pool("mla", [n], layers=1).check([subset(9, 100, 50) + list(range(39000, n))])


def test_accepted_paths():
    lens = [501, 640, 64]
    p = Pool("gqa", lens, spare=64, layers=4)
    p.check([[0, 3, 17, 40], [5], [0, 1, 2, 60, 61, 63]], first=lens, rotate=False)


def test_compact_offsets_beyond_32_bits():
    # a pool whose rows lie more than 2^32 bytes apart
    slots, d = 64 * 4, 576
    ss = (1 << 32) // 2 // 64 + 8
    flat = torch.empty(slots * ss + d, dtype=torch.bfloat16, device="cuda")
    row = flat.as_strided((1, slots, d), (slots * ss, ss, 1))
    row.copy_(torch.randn(1, slots, d, device="cuda").to(torch.bfloat16))
    old = row.clone()
    desc = kv.pool_desc(row[..., :512], row[..., 512:], 64, 1, 1e4)
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    keep = torch.tensor([list(range(100, 256))], dtype=torch.int32, device="cuda")
    count = torch.tensor([156], dtype=torch.int32, device="cuda")
    ws = kv.compact_workspace(desc, 1, 4, 156)
    kv.kv_compact(desc, table, None, keep, count, False, ws)
    assert kv.kv_get_device_status(ws) == kv.KV_OK
    slot = lambda p: table[0].long()[p // 64] * 64 + p % 64  # noqa: E731
    i = torch.arange(156, device="cuda")
    assert torch.equal(row[0, slot(i)], old[0, slot(i + 100)])
    assert torch.equal(row[0, slot(i[:100] + 156)], old[0, slot(i[:100] + 156)])


@pytest.mark.parametrize("bad", ["count", "low", "first", "order", "table", "block"])
def test_compact_reports_what_does_not_fit(bad):
    p = Pool("mla", [200, 200])
    keep = torch.tensor([subset(1, 200, 50), subset(2, 200, 50)], dtype=torch.int32)
    count = torch.tensor([50, 50], dtype=torch.int32)
    first = torch.zeros(2, dtype=torch.int32)
    table = p.table.clone()
    before = p.bits()
    if bad == "count":
        count[0] = 51
    elif bad == "low":
        count[0] = -1
    elif bad == "first":
        first[0] = -1
    elif bad == "order":
        keep[0, 49] = 3
    elif bad == "table":
        keep[0, 49] = 256
    elif bad == "block":
        table[0, 0] = 10 ** 6
    ws = kv.compact_workspace(p.desc, 2, 4, 50)
    kv.kv_compact(p.desc, table.cuda(), first.cuda(), keep.cuda(), count.cuda(), True, ws)
    assert kv.kv_get_device_status(ws) == kv.KV_ERR_OUT_OF_RANGE
    after = p.bits()
    s, i = 0, np.arange(50)
    if bad in ("count", "low", "first", "block"):  # the whole sequence stays
        for k in before:
            rows = p.slot(0, np.arange(200))
            assert np.array_equal(before[k][:, rows], after[k][:, rows])
    # the other sequence has moved
    src, dst = p.slot(1, keep[1].numpy().astype(np.int64)), p.slot(1, i)
    assert np.array_equal(after["copy"][:, dst], before["copy"][:, src])


def test_compact_wait_that_runs_out():
    p = Pool("mla", [2000], layers=3)
    keep = torch.arange(1, 2000, dtype=torch.int32, device="cuda")[None].contiguous()
    count = torch.tensor([1999], dtype=torch.int32, device="cuda")
    ws = kv.compact_workspace(p.desc, 1, p.table.shape[1], 1999)
    kv.kv_set_wait_limit_ns(2_000_000)
    kv.kv_set_splice_skip_publish(0)
    try:
        kv.kv_compact(p.desc, p.table.cuda(), None, keep, count, False, ws)
        assert kv.kv_get_device_status(ws) == kv.KV_ERR_TIMEOUT
    finally:
        kv.kv_set_splice_skip_publish(-1)
        kv.kv_set_wait_limit_ns(0)
    Pool("mla", [2000], layers=3).check([list(range(1, 2000))])


def test_captured_together():
    """Choice and move in one graph, replayed on new weights without the host."""
    p = Pool("mla", [500, 400])
    w = heavy(7, 2, 500).cuda()
    lens = torch.tensor([500, 400], dtype=torch.int32, device="cuda")
    budget = torch.tensor([200, 100], dtype=torch.int32, device="cuda")
    keep = torch.zeros(2, 200, dtype=torch.int32, device="cuda")
    count = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws, cws = kv.evict_workspace(2, 500), kv.compact_workspace(p.desc, 2, p.table.shape[1], 200)
    table = p.table.cuda()

    def step():
        kv.kv_evict_select(w, lens, budget, 4, 16, keep, count, None, ws)
        kv.kv_compact(p.desc, table, None, keep, count, False, cws)

    saved = {k: v.clone() for k, v in p.parts.items()}
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (8, 9):
        w.copy_(heavy(seed, 2, 500))
        for k, v in saved.items():
            p.parts[k].copy_(v)
        before = p.bits()
        g.replay()
        after = p.bits()
        want = ref_select(w.cpu(), [500, 400], [200, 100], 4, 16)
        for s in range(2):
            assert keep[s, : len(want[s])].tolist() == want[s]
            src, dst = p.slot(s, np.array(want[s])), p.slot(s, np.arange(len(want[s])))
            for k in before:
                assert np.array_equal(after[k][:, dst], before[k][:, src])
        assert kv.kv_get_device_status(cws) == kv.KV_OK


def test_select_long_and_alike():
    # more keys of one first digit than are listed; runs of more than 2^16 tokens in a block
    w = 1.0 + heavy(11, 2, 200000) * 1e-3
    w[1, ::2] = 1.25
    check_select(w, [200000, 199999], [70000, 33333], 4, 100)
    w = heavy(12, 80, 70000)
    check_select(w, [70000 - 7 * i for i in range(80)], [500 + i for i in range(80)], 0, 3)
    check_select(torch.zeros(2, 66000), [66000, 40000], [100, 39999], 1, 1)


def step_by_step(kind, quant):
    """One request under a bounded cache: attention, what its keys received, the choice, the
    move, and attention over what is left, against the same in 64 bits."""
    from _keep import Sums
    s = Sums(kind, [(3, 400), (1, 250)], 16 if kind == "mla" else 32, keep=0.0, quant=quant, seed=5)
    out, lse = s.run_attention()
    kv.kv_attention_weights(s.desc, s.layer, s.attn, s.q, lse, s.weights, 0.0, s.wws)
    lens = torch.tensor([400, 250], dtype=torch.int32, device="cuda")
    budget = torch.tensor([120, 250], dtype=torch.int32, device="cuda")
    keep, count = torch.zeros(2, 250, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    kept = torch.zeros(2, 250, device="cuda")
    ws = kv.evict_workspace(2, s.weights.shape[1])
    kv.kv_evict_select(s.weights, lens, budget, 4, 32, keep, count, kept, ws)
    table = s.table.cuda()
    cws = kv.compact_workspace(s.desc, 2, table.shape[1], 250)
    before = [getattr(s.pool, n)[s.layer].clone() for n in ("copy", "rot")]
    kv.kv_compact(s.desc, table, None, keep, count, False, cws)
    assert [kv.kv_get_device_status(w) for w in (s.wws, ws, cws)] == [kv.KV_OK] * 3
    want = ref_select(s.weights.cpu(), [400, 250], [120, 250], 4, 32)
    assert count.tolist() == [120, 250]
    for q in range(2):
        assert keep[q, : len(want[q])].tolist() == want[q]
        src, dst = s.slots(q)[want[q]].cuda(), s.slots(q)[: len(want[q])].cuda()
        for part, old in zip(("copy", "rot"), before):
            new = getattr(s.pool, part)[s.layer]
            v = torch.uint8 if new.element_size() == 1 else torch.int16
            assert torch.equal(new.view(v)[dst], old.view(v)[src])
    # the kept keys' attention: their shares of the whole context's, which sum to what is kept
    attn = kv.attn_desc(s.attn._tensors[0], count, table, 3, 250, s.scale)
    lse2 = torch.empty_like(lse)
    kv.kv_attention(s.desc, s.layer, attn, s.q, out, lse2, kv.attn_workspace(s.desc, attn, s.q))
    share = torch.exp(lse2 - lse)  # of each row's weight that the kept keys hold
    rows = [share[:3].sum(), share[3:].sum()]
    for q in range(2):
        assert abs(float(kept[q, : count[q]].sum()) - float(rows[q])) < 1e-3 * float(rows[q])


@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", False), ("gqa", True), ("mla", True)])
def test_a_bounded_cache_step_by_step(kind, quant):
    step_by_step(kind, quant)


@pytest.mark.parametrize("kind,quant", [("mla", False), ("gqa", True)])
def test_drafted_tokens_are_verified_and_close_up(kind, quant):
    """A tree's path that is accepted has the results of the same tokens as a causal chunk, and
    closes up into the cache that they would have left."""
    from _keep import Tree
    parents = [-1, 0, 0, 1, 3, 2, 3, 6]
    path = [0, 1, 3, 6, 7]
    sees = []
    for j, up in enumerate(parents):
        sees.append((sees[up] if up >= 0 else 0) | 1 << j)
    assert torch.equal(kv.tree_mask([parents], "cpu")[:, 0], torch.tensor(sees, dtype=torch.int32))
    t = Tree(kind, [(8, 208)], 16 if kind == "mla" else 32, masks=[sees], quant=quant, seed=6)
    out, lse = t.check()
    out, lse = out[path].clone(), lse[path].clone()
    table = t.table.cuda()
    first = torch.tensor([200], dtype=torch.int32, device="cuda")
    keep = torch.tensor([path], dtype=torch.int32, device="cuda")
    count = torch.tensor([5], dtype=torch.int32, device="cuda")
    ws = kv.compact_workspace(t.desc, 1, table.shape[1], 5)
    kv.kv_compact(t.desc, table, first, keep, count, False, ws)
    assert kv.kv_get_device_status(ws) == kv.KV_OK
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    attn = kv.attn_desc(off, torch.tensor([205], dtype=torch.int32, device="cuda"), table, 5, 205, t.scale)
    q = t.q[path].contiguous()
    got, glse = torch.empty_like(out), torch.empty_like(lse)
    kv.kv_attention(t.desc, t.layer, attn, q, got, glse, kv.attn_workspace(t.desc, attn, q))
    # both are within the bounds of Batch.reference of the same numbers
    _, _, to, tl = t.reference()
    assert not ((got.double() - out.double()).abs() > 2 * to[path]).any()
    assert not ((glse.double() - lse.double()).abs() > 2 * tl[path]).any()
