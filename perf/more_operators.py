"""Cases of the operators that a serving loop needs around attention when it drafts
tokens or bounds its cache: attention of a tree of drafted tokens (``tree``), what
each cached key has received of the queries' attention (``weights``), the choice of
the tokens that stay (``select``) and the move of their rows together (``compact``;
also of the rows of an accepted path).

``run`` computes a case in plain torch, or through the library where ``own`` is
set; ``exact`` computes the same outputs in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

# Row shapes of the library's pools: (width of the verbatim part, rotary heads,
# rotary head dim, RoPE base).
KINDS = {
    "mla": (512, 1, 64, 10000.0),
    "gqa": (1024, 8, 128, 500000.0),
    "gqa4": (512, 4, 128, 1000000.0),
    "mha": (4096, 32, 128, 10000.0),
}
GROUP = 128  # elements that share one scale of a quantised row


def listed():
    t, w, c = "tree", "weights", "compact"
    return [
        # one request, a small tree, short context: the smallest call
        dict(name="tree, GQA, 16 over 577", op=t, kind="gqa", heads=32, seqs=1, q_lo=16, q_hi=16,
             kv_lo=577, kv_hi=577, block=64, quant=False),
        # a batch of requests that verify their drafts, ragged trees and contexts
        dict(name="tree, GQA, 16 ragged", op=t, kind="gqa", heads=32, seqs=16, q_lo=26, q_hi=64,
             kv_lo=1030, kv_hi=16384, block=64, quant=False),
        # drafts over quantised latent rows
        dict(name="tree, MLA e4m3, 8 ragged", op=t, kind="mla", heads=16, seqs=8, q_lo=25, q_hi=61,
             kv_lo=2049, kv_hi=8192, block=64, quant=True),
        # one request counts its step's attention: latency
        dict(name="weights, GQA, 1 x 577", op=w, kind="gqa", heads=32, seqs=1, q_lo=1, q_hi=1,
             kv_lo=577, kv_hi=577, block=64, quant=False, causal=True, window=0, sinks=0, keep=1.0),
        # a decode batch over the quantised pool: the keys are read once
        dict(name="weights, GQA e4m3, 64 ragged", op=w, kind="gqa", heads=32, seqs=64, q_lo=1,
             q_hi=1, kv_lo=301, kv_hi=16384, block=64, quant=True, causal=True, window=0, sinks=0,
             keep=1.0),
        # a decode batch over latent rows, 128 heads to each, older steps fading
        dict(name="weights, MLA, 32 ragged", op=w, kind="mla", heads=128, seqs=32, q_lo=1, q_hi=1,
             kv_lo=2049, kv_hi=16384, block=64, quant=False, causal=True, window=0, sinks=0,
             keep=0.95),
        # every query of a prompt chunk counts: bound by the tensor cores
        dict(name="weights, GQA, 4096 over 16384", op=w, kind="gqa", heads=32, seqs=1, q_lo=4096,
             q_hi=4096, kv_lo=16384, kv_hi=16384, block=64, quant=False, causal=True, window=0,
             sinks=0, keep=0.0),
        # half of each context of a decode batch is to stay
        dict(name="select, 64 ragged", op="select", seqs=64, kv_lo=301, kv_hi=16384, share=0.5,
             sinks=4, recent=64),
        # one long context down to a fixed budget
        dict(name="select, 8192 of 131072", op="select", seqs=1, kv_lo=131072, kv_hi=131072,
             share=0.0625, sinks=4, recent=128),
        # accepted drafts close up behind their contexts, every layer: latency
        dict(name="accept, MLA, 32 paths", op=c, kind="mla", layers=61, seqs=32, kv_lo=501,
             kv_hi=2048, first=True, share=0.0, path=6, nodes=61, block=64, quant=False,
             rotate=False),
        # the kept half of quantised latent rows closes up, k_pe turned to its new positions
        dict(name="evict, MLA e4m3, 4 x 16384", op=c, kind="mla", layers=61, seqs=4, kv_lo=9001,
             kv_hi=16384, first=False, share=0.5, path=0, nodes=0, block=64, quant=True,
             rotate=True),
        # head rows down to two fifths, every K head turned
        dict(name="evict, GQA, 4 x 8192", op=c, kind="gqa", layers=32, seqs=4, kv_lo=5003,
             kv_hi=8192, first=False, share=0.4, path=0, nodes=0, block=64, quant=False,
             rotate=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "weights", "weights", "select", "compact", "compact"])
    if op == "select":
        kv = _log(rng, 16, 131072)
        return dict(op=op, seqs=max(1, min(_log(rng, 1, 64), (1 << 21) // kv)),
                    kv_lo=max(1, kv // 3), kv_hi=kv, share=math.exp(rng.uniform(math.log(0.02), 0)),
                    sinks=rng.choice([0, 1, 4, 67]), recent=rng.choice([0, 1, 64, 511]))
    kind = rng.choice(sorted(KINDS))
    cd, h, d, _ = KINDS[kind]
    quant = rng.random() < 0.4
    if op == "compact":
        layers, seqs, kv = _log(rng, 1, 61), _log(rng, 1, 64), _log(rng, 32, 32768)
        while seqs > 1 and seqs * kv * layers * (cd + h * d) > 1 << 31:
            seqs = seqs * 2 // 3
        while seqs * kv * layers * (cd + h * d) > 1 << 31:
            layers = layers * 2 // 3
        path = rng.random() < 0.3
        nodes = _log(rng, 2, 64)
        return dict(op=op, kind=kind, layers=layers, seqs=seqs, kv_lo=max(1, kv // 2), kv_hi=kv,
                    first=path, share=0.0 if path else math.exp(rng.uniform(math.log(0.05), 0)),
                    path=max(1, nodes // 4) if path else 0, nodes=nodes if path else 0,
                    block=rng.choice([16, 64]), quant=quant,
                    rotate=not path and (not quant or kind == "mla") and rng.random() < 0.7)
    heads = {"mla": rng.choice([16, 32, 64, 128]), "gqa": rng.choice([8, 32, 40, 64]),
             "gqa4": rng.choice([4, 16, 28]), "mha": 32}[kind]
    seqs, kv = _log(rng, 1, 64), _log(rng, 16, 32768)
    q = _log(rng, 1, 128 if op == "tree" else 4096)
    if op == "weights" and rng.random() < 0.5:
        q = 1
    kv = max(kv, q)
    wide = 4 if kind == "mla" else 1
    while seqs > 1 and (seqs * heads * q * kv * wide > 32 * 4096 * 16384 // 2 or
                        seqs * kv * h * d > 1 << 29):
        seqs = seqs * 2 // 3
    while seqs * heads * q * kv * wide > 32 * 4096 * 16384 // 2:
        q = max(1, q * 2 // 3)
    case = dict(op=op, kind=kind, heads=heads, seqs=seqs, q_lo=max(1, q // 2), q_hi=q,
                kv_lo=max(q, kv // 3), kv_hi=kv, block=rng.choice([16, 64]), quant=quant)
    if op == "weights":
        win = rng.random() < 0.25
        case.update(causal=win or rng.random() < 0.8, window=_log(rng, 64, 8192) if win else 0,
                    sinks=rng.choice([0, 1, 4, 67]) if win else 0, keep=rng.choice([0.0, 1.0, 0.95]))
    return case


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _kv_lengths(case):
    r, n = _rng(case), case["seqs"]
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(n)]
    kv[-1] = case["kv_hi"]
    return kv


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    r, n = _rng(case), case["seqs"]
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    kv = [max(a, r.randint(case["kv_lo"], case["kv_hi"])) for a in q]
    q[-1], kv[-1] = case["q_hi"], case["kv_hi"]
    return q, kv


def _kept(case):
    """Rows that stay, of each sequence of a compaction."""
    if case["first"]:
        r = _rng(case)
        n = [r.randint(1, case["path"]) for _ in range(case["seqs"])]
        n[-1] = case["path"]
        return n
    return [max(1, int(case["share"] * k)) for k in _kv_lengths(case)]


def _pairs(case, nq, nk):
    """Visible (query, key) pairs of one head of one sequence, and the keys that any query sees."""
    i = torch.arange(nq)
    p = nk - nq + i
    hi = torch.where(torch.tensor(case["causal"]), p + 1, torch.full_like(p, nk))
    if not case["window"]:
        return int(hi.sum()), nk
    lo = (p - case["window"] + 1).clamp(min=0)
    sinks = torch.minimum(torch.full_like(lo, case["sinks"]), lo)
    seen = nk - int(lo[0]) + min(case["sinks"], int(lo[0]))
    return int((hi - lo + sinks).sum()), seen


def work(case):
    if case["op"] == "select":
        kv = _kv_lengths(case)
        kept = sum(max(1, int(case["share"] * k)) for k in kv)
        return {"bytes": 4 * sum(kv) + 8 * kept + 12 * case["seqs"], "flops": 2 * sum(kv)}
    cd, h, d, _ = KINDS[case["kind"]]
    mla, q8 = case["kind"] == "mla", case["quant"]
    rot = 2 * d if mla or not q8 else d + 4  # bytes of a rotary head
    copy = cd + cd // GROUP * 4 if q8 else 2 * cd
    if case["op"] == "compact":
        rows = sum(_kept(case))
        if not case["first"]:  # rows of the longest unbroken start stay where they are
            r = min(case["share"], 0.999)
            rows = max(0, rows - int(case["seqs"] * r / (1 - r)))
        n = rows * case["layers"]
        return {"bytes": 2 * n * (copy + h * rot) + 4 * rows,
                "flops": 3 * n * h * d if case["rotate"] else 0}
    dk, dv = (cd + d, cd) if mla else (d, d)
    q, kv = _lengths(case)
    tokens, heads = sum(q), case["heads"]
    if case["op"] == "tree":
        pairs = sum(a * (b - a) + a * 6 for a, b in zip(q, kv))  # some six ancestors to a token
        words = -(-max(q) // 32)
        return {"bytes": tokens * heads * (2 * (dk + dv) + 4) + sum(kv) * (copy + h * rot) +
                4 * tokens * words, "flops": 2 * (dk + dv) * heads * pairs}
    seen = [_pairs(case, a, b) for a, b in zip(q, kv)]
    key = copy + rot if mla else h * rot
    sums = sum(kv) * (8 if case["keep"] else 4)
    return {"bytes": tokens * heads * (2 * dk + 4) + sum(s for _, s in seen) * key + sums,
            "flops": 2 * dk * heads * sum(p for p, _ in seen)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(g, shape):
    """Cache rows: unit normal, every 16th channel six times as large, as the
    keys and latents of trained models have a few channels that stand out."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x[..., ::16] *= 6.0
    return x.to(torch.bfloat16)


def _quantize(x):
    """e4m3 values and scales: 2^e with the smallest e that keeps a group's largest
    magnitude at or below 448."""
    y = x.float().unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(y.abs().amax(-1))
    e = torch.where(m == 0, 0, (e - 9 + (m > 0.875)).clamp(min=-120))
    one = torch.ones_like(m)
    return ((y * torch.ldexp(one, -e).unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2),
            torch.ldexp(one, e))


def _pool(g, kind, layers, slots, quant):
    """Tensors of a pool in the library's layout."""
    cd, h, d, _ = KINDS[kind]
    if not quant:
        if kind == "mla":
            row = torch.empty(layers, slots, cd + d, device="cuda", dtype=torch.bfloat16)
            for l in range(layers):
                row[l] = _rows(g, (slots, cd + d))
            return {"copy": row[..., :cd], "rot": row[..., cd:]}
        p = {k: torch.empty(layers, slots, w, device="cuda", dtype=torch.bfloat16)
             for k, w in (("copy", cd), ("rot", h * d))}
        for l in range(layers):
            p["copy"][l], p["rot"][l] = _rows(g, (slots, cd)), _rows(g, (slots, h * d))
        return p
    f8, f4 = torch.float8_e4m3fn, torch.float32
    z = lambda w, t: torch.empty(layers, slots, w, device="cuda", dtype=t)  # noqa: E731
    p = {"copy": z(cd, f8), "copy_scale": z(cd // GROUP, f4)}
    if kind == "mla":
        p["rot"] = z(d, torch.bfloat16)
    else:
        p["rot"], p["rot_scale"] = z(h * d, f8), z(h * d // GROUP, f4)
    for l in range(layers):
        p["copy"][l], p["copy_scale"][l] = _quantize(_rows(g, (slots, cd)))
        r = _rows(g, (slots, h * d))
        if kind == "mla":
            p["rot"][l] = r
        else:
            p["rot"][l], p["rot_scale"][l] = _quantize(r)
    return p


def _desc(kv, case, p):
    _, h, _, base = KINDS[case["kind"]]
    if case["quant"]:
        return kv.quant_pool_desc(p["copy"], p["copy_scale"], p["rot"], p.get("rot_scale"),
                                  case["block"], h)
    return kv.pool_desc(p["copy"], p["rot"], case["block"], h, base)


def _trees(case, ql):
    """Masks of drafted trees: token 0 is the last accepted one, every other hangs on
    an earlier one, near the root more often, and sees itself and its ancestors."""
    r, words = _rng(case), -(-max(ql) // 32)
    rows = []
    for n in ql:
        sees = []
        for j in range(n):
            up = sees[int(j * r.random() ** 2)] if j else 0
            sees.append(up | 1 << j)
        rows += sees
    bits = [[(x >> 32 * w) & 0xFFFFFFFF for w in range(words)] for x in rows]
    return torch.tensor(bits, dtype=torch.int64).to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "select":
        kl = _kv_lengths(case)
        n, most = case["seqs"], case["kv_hi"]
        # heavy-tailed sums; some tokens were never seen and tie at zero, some others tie too
        x = torch.randn(n, most, generator=g, device="cuda").mul_(2.0).exp_()
        u = torch.rand(n, most, generator=g, device="cuda")
        x = torch.where(u < 0.05, 0.0, torch.where(u < 0.1, torch.round(x * 8) / 8, x))
        s["weights"] = x
        s["kv_len"] = torch.tensor(kl, dtype=torch.int32).cuda()
        s["budget"] = torch.tensor([max(1, int(case["share"] * k)) for k in kl],
                                   dtype=torch.int32).cuda()
        s["most"] = max(1, int(case["share"] * most))
        s["keep"] = torch.zeros(n, s["most"], dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros(n, s["most"], device="cuda")
        if own:
            import position_independent_mla_gb300 as kv
            s["ws"] = kv.evict_workspace(n, most)
        return s
    b, n = case["block"], case["seqs"]
    if case["op"] == "compact":
        kl, kept = _kv_lengths(case), _kept(case)
        spare = case["nodes"] if case["first"] else 0
        per = -(-(max(kl) + spare) // b)
        s["keep"] = torch.zeros(n, max(kept), dtype=torch.int32, device="cuda")
        for i, (a, c) in enumerate(zip(kl, kept)):
            many = case["nodes"] if case["first"] else a
            c = min(c, many)
            s["keep"][i, :c] = torch.randperm(many, generator=g, device="cuda")[:c].sort()[0].int()
        s["count"] = torch.tensor(kept, dtype=torch.int32).cuda()
        s["first"] = torch.tensor(kl, dtype=torch.int32).cuda() if case["first"] else None
        s["most"], layers = max(kept), case["layers"]
    else:
        ql, kl = _lengths(case)
        per, layers = -(-max(kl) // b), 2
    blocks = n * per + 3
    s["table"] = torch.randperm(blocks, generator=g, device="cuda")[: n * per].int().view(n, per)
    s["pool"] = _pool(g, case["kind"], layers, blocks * b, case["quant"])
    if own:
        import position_independent_mla_gb300 as kv
        s["pd"] = _desc(kv, case, s["pool"])
    if case["op"] == "compact":
        if own:
            s["ws"] = kv.compact_workspace(s["pd"], n, per, s["most"])
        return s
    cd, h, d, _ = KINDS[case["kind"]]
    mla = case["kind"] == "mla"
    s["layer"] = 1
    off = torch.tensor([0] + ql).cumsum(0)
    s["q_off"], s["kv_len"] = off.int().cuda(), torch.tensor(kl, dtype=torch.int32).cuda()
    tokens = int(off[-1])
    s["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(ql)).cuda()
    s["idx"] = torch.arange(tokens).cuda() - s["q_off"].long()[s["seq"]]
    s["max_q"], s["max_kv"] = max(ql), max(kl)
    dk, dv = (cd + d, cd) if mla else (d, d)
    s["scale"] = 192 ** -0.5 if mla else 128 ** -0.5
    s["query"] = torch.randn(tokens, case["heads"], dk, generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "tree":
        s["mask"] = _trees(case, ql)
        s["out"] = torch.empty(tokens, case["heads"], dv, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.empty(tokens, case["heads"], device="cuda")
    else:  # what attention over the same keys has left, and the weights of earlier steps
        s["lse"] = _by_token(s, torch.logsumexp(_scores(s), -1)).contiguous()
        s["weights"] = torch.rand(n, s["max_kv"], generator=g, device="cuda")
    if own:
        more = {} if case["op"] == "tree" else dict(causal=case["causal"], window=case["window"],
                                                    sinks=case["sinks"])
        s["ad"] = kv.attn_desc(s["q_off"], s["kv_len"], s["table"], max_q_len=s["max_q"],
                               max_kv_len=s["max_kv"], scale=s["scale"], **more)
        s["ws"] = (kv.tree_workspace if case["op"] == "tree" else kv.weights_workspace)(
            s["pd"], s["ad"], s["query"])
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def _value(x8, scale):
    y = x8.float()
    if scale is None:
        return y
    return (y.unflatten(-1, (-1, GROUP)) * scale.unsqueeze(-1)).flatten(-2)


def _at(t, layer, slots):
    """Rows of a layer at the slots (8-bit values are indexed as bytes)."""
    if t is None:
        return None
    return (t[layer].view(torch.uint8)[slots].view(t.dtype) if t.dtype == torch.float8_e4m3fn
            else t[layer][slots])


def _heads(s, name):
    """[S, K, heads, width] of one part of the cached rows, in fp32."""
    k = torch.arange(s["max_kv"], device="cuda")
    b, p = s["case"]["block"], s["pool"]
    slots = s["table"].long()[:, k // b] * b + k % b
    x = _value(_at(p[name], s["layer"], slots), _at(p.get(name + "_scale"), s["layer"], slots))
    mla = s["case"]["kind"] == "mla"
    return x.unsqueeze(2) if mla else x.unflatten(-1, (-1, 128))


def _scores(s):
    """[S, key heads, group, Q, K], -inf where a query does not see a key."""
    case = s["case"]
    h = KINDS[case["kind"]][1]
    nq, nk, heads = s["max_q"], s["max_kv"], case["heads"]
    key = _heads(s, "rot")
    if case["kind"] == "mla":
        key = torch.cat([_heads(s, "copy"), key], -1)
    q = torch.zeros(case["seqs"], nq, heads, s["query"].shape[-1], device="cuda")
    q[s["seq"], s["idx"]] = s["query"].float()
    q = q.unflatten(2, (h, heads // h)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [S, h, g*nq, d]
    score = (q @ key.permute(0, 2, 3, 1)).mul_(s["scale"]).unflatten(2, (heads // h, nq))
    k, i = torch.arange(nk, device="cuda"), torch.arange(nq, device="cuda")
    length = s["kv_len"].long()[:, None, None]
    new = (s["q_off"][1:] - s["q_off"][:-1]).long()[:, None, None]
    real = i[None, :, None] < new  # rows of longer sequences' queries
    see = (k < length) & real
    if case["op"] == "tree":
        j = (k - (length - new)).expand(-1, nq, -1)  # which new token key k is
        m = torch.zeros(case["seqs"], nq, s["mask"].shape[1], dtype=torch.int64, device="cuda")
        m[s["seq"], s["idx"]] = s["mask"].long() & 0xFFFFFFFF
        c = j.clamp(0, nq - 1)
        see = see & ((j < 0) | (m.gather(2, c // 32) >> (c % 32) & 1).bool())
    else:
        pos = length - new + i[None, :, None]
        if case["causal"]:
            see = see & (k <= pos)
        if case["window"]:
            see = see & ((k > pos - case["window"]) | (k < case["sinks"]))
    return score.masked_fill_(~see[:, None, None], -math.inf)


def _by_token(s, x):
    """[S, h, group, Q, ...] -> [token, head, ...]."""
    x = x.movedim(3, 1).flatten(2, 3)
    return x[s["seq"], s["idx"]]


def _tree(s):
    score = _scores(s)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1)
    val = _heads(s, "copy")
    out = (p.flatten(2, 3) @ val.permute(0, 2, 1, 3)).unflatten(2, p.shape[2:4])
    out = out / total.clamp(min=1e-38).unsqueeze(-1)
    return _by_token(s, out).to(torch.bfloat16), _by_token(s, total.log() + top.squeeze(-1))


def _weights(s):
    case = s["case"]
    h = KINDS[case["kind"]][1]
    lse = torch.zeros(case["seqs"], s["max_q"], case["heads"], device="cuda")
    lse[s["seq"], s["idx"]] = s["lse"]
    lse = lse.unflatten(2, (h, -1)).permute(0, 2, 3, 1)
    lse = torch.where(lse == -math.inf, torch.full_like(lse, math.inf), lse)
    new = _scores(s).sub_(lse.unsqueeze(-1)).exp_().sum((1, 2, 3))
    old = s["weights"]
    k = torch.arange(s["max_kv"], device="cuda")
    new = case["keep"] * old + new if case["keep"] else new
    s["weights"] = torch.where(k < s["kv_len"].long()[:, None], new, old)
    return s["weights"]


def _select(s):
    case, w = s["case"], s["weights"]
    k = torch.arange(w.shape[1], device="cuda")
    length, budget = s["kv_len"].long()[:, None], s["budget"].long()[:, None]
    # sinks first, then the last tokens from the end, then by weight, the lowest index first
    rank = torch.where(w == w, w, torch.full_like(w, -math.inf)).double()
    rank = torch.where(k >= length - case["recent"], 1e300 + (k + 1.0) * 1e290, rank)
    rank = torch.where(k < case["sinks"], torch.full_like(rank, math.inf), rank)
    rank = torch.where(k < length, rank, torch.full_like(rank, -math.inf))
    # (NaN and -inf share a rank, before what lies past the end: the sort is stable)
    order = torch.sort(rank, dim=1, descending=True, stable=True)[1]
    count = torch.minimum(length, budget)
    keep = torch.where(k < count, order, torch.full_like(order, w.shape[1])).sort(1)[0]
    at = torch.arange(s["most"], device="cuda") < count
    keep = keep[:, : s["most"]].clamp(max=w.shape[1] - 1)
    s["keep"] = torch.where(at, keep.int(), s["keep"])
    s["kept"] = torch.where(at, w.gather(1, keep), s["kept"])
    s["count"] = count[:, 0].int()
    return s["keep"], s["count"], s["kept"]


def _slots(s):
    """Slots that rows move from and to, and by how many positions, of every sequence."""
    b, first = s["case"]["block"], s["first"]
    i = torch.arange(s["most"], device="cuda")
    there = i < s["count"].long()[:, None]
    base = 0 if first is None else first.long()[:, None]
    src, dst = base + s["keep"].long(), (base + i).expand_as(there)
    seq = torch.arange(len(s["count"]), device="cuda")[:, None].expand_as(src)[there]
    src, dst = src[there], dst[there]
    slot = lambda p: s["table"].long()[seq, p // b] * b + p % b  # noqa: E731
    return slot(src), slot(dst), dst - src


def _turn(x, shift, dim, base):
    """R(shift) of rows x [L, N, heads*dim]; the angles in 64 bits, the turn in 32."""
    j = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
    a = shift.double()[:, None] * base ** (-2.0 * j / dim)
    c, n = a.cos().float()[:, None], a.sin().float()[:, None]
    u, v = x.float().unflatten(-1, (-1, 2, dim // 2)).unbind(-2)
    return torch.stack([u * c - v * n, u * n + v * c], -2).flatten(-3).to(x.dtype)


def _compact(s):
    case, p = s["case"], s["pool"]
    _, _, d, base = KINDS[case["kind"]]
    src, dst, shift = _slots(s)
    for name, t in p.items():
        t = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
        x = t[:, src]
        if name == "rot" and case["rotate"]:
            x = torch.where((shift == 0)[:, None], x, _turn(x, shift, d, base))
        t[:, dst] = x
    return p


def run(s):
    case = s["case"]
    if own:
        import position_independent_mla_gb300 as kv
        if case["op"] == "tree":
            kv.kv_tree_attention(s["pd"], s["layer"], s["ad"], s["mask"], s["query"], s["out"],
                                 s["lse"], s["ws"])
            return s["out"], s["lse"]
        if case["op"] == "weights":
            kv.kv_attention_weights(s["pd"], s["layer"], s["ad"], s["query"], s["lse"],
                                    s["weights"], case["keep"], s["ws"])
            return s["weights"]
        if case["op"] == "select":
            kv.kv_evict_select(s["weights"], s["kv_len"], s["budget"], case["sinks"],
                               case["recent"], s["keep"], s["count"], s["kept"], s["ws"])
            return s["keep"], s["count"], s["kept"]
        more = dict(rope_base=KINDS[case["kind"]][3]) if case["quant"] else {}
        kv.kv_compact(s["pd"], s["table"], s["first"], s["keep"], s["count"], case["rotate"],
                      s["ws"], **more)
        return s["pool"]
    return {"tree": _tree, "weights": _weights, "select": _select, "compact": _compact}[
        case["op"]](s)


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_rows(s, q, nk):
    """Both parts of one sequence's cached rows, in double precision."""
    b, l, part = s["case"]["block"], s["layer"], {}
    pos = torch.arange(nk, device="cuda")
    slot = s["table"][q].long()[pos // b] * b + pos % b
    for name in ("copy", "rot"):
        x = s["pool"][name][l].to(torch.float32)[slot].double()
        sc = s["pool"].get(name + "_scale")
        part[name] = x if sc is None else x * sc[l][slot].double().repeat_interleave(GROUP, -1)
    return part


def _exact_attention(s):
    case = s["case"]
    cd, h, d, _ = KINDS[case["kind"]]
    mla, heads = case["kind"] == "mla", case["heads"]
    tree = case["op"] == "tree"
    ql, kl = _lengths(case)
    f8 = dict(device="cuda", dtype=torch.float64)
    out, lse = torch.empty(sum(ql), heads, cd if mla else d, **f8), torch.empty(sum(ql), heads, **f8)
    sums = s["weights"].double() if not tree else None
    at = 0
    for q, (nq, nk) in enumerate(zip(ql, kl)):
        part = _exact_rows(s, q, nk)
        far = nk - nq + torch.arange(nq, device="cuda")[:, None] - torch.arange(nk, device="cuda")
        if tree:
            ok = torch.zeros(nq, nk, dtype=torch.bool, device="cuda")
            ok[:, : nk - nq] = True
            for j in range(nq):
                ok[:, nk - nq + j] = (s["mask"][at:at + nq, j // 32] >> j % 32) & 1 == 1
        else:
            ok = torch.ones_like(far, dtype=torch.bool) if not case["causal"] else far >= 0
            if case["window"]:
                sink = torch.arange(nk, device="cuda") < case["sinks"]
                ok = ok & ((far < case["window"]) | sink)
            sums[q, :nk] = sums[q, :nk] * case["keep"] if case["keep"] else 0.0
        bias = torch.where(ok, 0.0, -math.inf).double()
        for head in range(heads):
            j = head // (heads // h)
            key = torch.cat([part["copy"], part["rot"]], 1) if mla else part["rot"][:, j * d:j * d + d]
            z = s["query"][at:at + nq, head].double() @ key.T * s["scale"] + bias
            if not tree:
                n = s["lse"][at:at + nq, head].double()
                sums[q, :nk] += torch.exp(z - torch.where(n == -math.inf, 0.0, n)[:, None]).sum(0)
                continue
            n = torch.logsumexp(z, -1)
            lse[at:at + nq, head] = n
            val = part["copy"] if mla else part["copy"][:, j * d:j * d + d]
            out[at:at + nq, head] = torch.exp(z - torch.where(n == -math.inf, 0.0, n)[:, None]) @ val
        at += nq
    return (out, lse) if tree else sums


def _exact_compact(s):
    case = s["case"]
    _, h, d, base = KINDS[case["kind"]]
    b = case["block"]
    keep, count, table = s["keep"].tolist(), s["count"].tolist(), s["table"].tolist()
    first = [0] * len(count) if s["first"] is None else s["first"].tolist()
    src, dst, shift = [], [], []
    for q, n in enumerate(count):
        for i in range(n):
            x, y = first[q] + keep[q][i], first[q] + i
            src.append(table[q][x // b] * b + x % b)
            dst.append(table[q][y // b] * b + y % b)
            shift.append(y - x)
    src, dst = torch.tensor(src).cuda(), torch.tensor(dst).cuda()
    got = {}
    for name, t in s["pool"].items():
        y = torch.empty(t.shape, device="cuda", dtype=torch.float32)
        for l in range(case["layers"]):  # what moves is exact in fp32; what turns is rounded to it
            y[l] = t[l].float()
            x = y[l][src]
            if name == "rot" and case["rotate"]:
                a = torch.tensor(shift).double().cuda()[:, None] * torch.tensor(
                    [base ** (-2.0 * f / d) for f in range(d // 2)], dtype=torch.float64).cuda()
                z = torch.polar(torch.ones_like(a), a)[:, None]
                w = x.double().view(-1, h, 2, d // 2)
                w = torch.complex(w[:, :, 0], w[:, :, 1]) * z
                x = torch.cat([w.real, w.imag], -1).reshape(-1, h * d).float()
            y[l][dst] = x
        got[name] = y
    return got


def _exact_select(s):
    case = s["case"]
    keep, kept = s["keep"].clone(), s["kept"].double()
    count = []
    for q, (n, b) in enumerate(zip(s["kv_len"].tolist(), s["budget"].tolist())):
        w = s["weights"][q, :n].tolist()
        near = max(min(case["sinks"], n), n - case["recent"])
        order = list(range(min(case["sinks"], n))) + list(range(n - 1, near - 1, -1))
        order += sorted(range(min(case["sinks"], n), near),
                        key=lambda i: (-w[i] if w[i] == w[i] else math.inf, i))
        mine = sorted(order[:b])
        count.append(len(mine))
        keep[q, : len(mine)] = torch.tensor(mine, dtype=torch.int32)
        kept[q, : len(mine)] = torch.tensor([w[i] for i in mine], dtype=torch.float64)
    return keep, torch.tensor(count, dtype=torch.int32).cuda(), kept


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(s)
    return _exact_compact(s) if case["op"] == "compact" else _exact_attention(s)
