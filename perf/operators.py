"""Cases of the serving operators over the paged cache: rows quantised as they
are written (``quantize``) and read back (``dequantize``), and attention of new
tokens over the cache (``attention``), with a sliding window and sink tokens
(``window``).

``run`` computes a case in plain torch, or through the library where ``own`` is
set; ``exact`` computes the same outputs in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

# Row shapes of the library's pools: (width of the verbatim part, rotary heads,
# rotary head dim, RoPE base, pairs of (key width, value width) that attention reads).
KINDS = {
    "mla": (512, 1, 64, 10000.0),
    "gqa": (1024, 8, 128, 500000.0),
    "gqa4": (512, 4, 128, 1000000.0),
    "mha": (4096, 32, 128, 10000.0),
}
GROUP = 128  # elements that share one scale


def listed():
    a, w = "attention", "window"
    return [
        # a decode step writes one layer's new rows of 32 requests: latency
        dict(name="write step, MLA, 32 rows", op="quantize", kind="mla", layers=1, rows=32,
             slots=8192),
        # a prefilled prompt goes into the quantised pool, every layer at once
        dict(name="write prompt, GQA, 16411 rows", op="quantize", kind="gqa", layers=32,
             rows=16411, slots=20480),
        # one registry chunk is read back for relocation, all 61 layers
        dict(name="read chunk, MLA, 1152 rows", op="dequantize", kind="mla", layers=61,
             rows=1152, slots=8192),
        # the registry chunks of a batch of requests, MHA rows
        dict(name="read chunks, MHA, 9001 rows", op="dequantize", kind="mha", layers=16,
             rows=9001, slots=16384),
        # one request, one new token, short context: the smallest call
        dict(name="decode, GQA, 1 x 577", op=a, kind="gqa", heads=32, seqs=1, q_lo=1, q_hi=1,
             kv_lo=577, kv_hi=577, block=64, quant=False, causal=True, window=0, sinks=0),
        # a decode batch of ragged contexts over the quantised pool
        dict(name="decode, GQA e4m3, 64 ragged", op=a, kind="gqa", heads=32, seqs=64, q_lo=1,
             q_hi=1, kv_lo=301, kv_hi=16384, block=64, quant=True, causal=True, window=0, sinks=0),
        # a prompt chunk after a relocated context: bound by the tensor cores
        dict(name="prefill, GQA, 4096 over 16384", op=a, kind="gqa", heads=32, seqs=1, q_lo=4096,
             q_hi=4096, kv_lo=16384, kv_hi=16384, block=64, quant=False, causal=True, window=0,
             sinks=0),
        # ragged chunks of a batch, seven query heads to a key head, quantised pool
        dict(name="chunks, GQA-4 e4m3, 8 ragged", op=a, kind="gqa4", heads=28, seqs=8, q_lo=57,
             q_hi=513, kv_lo=1030, kv_hi=8195, block=64, quant=True, causal=True, window=0,
             sinks=0),
        # a decode batch over latent rows, 128 heads sharing each row
        dict(name="decode, MLA, 32 ragged", op=a, kind="mla", heads=128, seqs=32, q_lo=1, q_hi=1,
             kv_lo=2049, kv_hi=16384, block=64, quant=False, causal=True, window=0, sinks=0),
        # short chunks (a question after a cached document) over quantised latent rows
        dict(name="chunks, MLA e4m3, 4 ragged", op=a, kind="mla", heads=16, seqs=4, q_lo=61,
             q_hi=350, kv_lo=4100, kv_hi=8192, block=64, quant=True, causal=True, window=0,
             sinks=0),
        # long contexts decoded through a window with sinks, 16-token blocks
        dict(name="window decode, MHA, 8 x 32768", op=w, kind="mha", heads=32, seqs=8, q_lo=1,
             q_hi=1, kv_lo=30011, kv_hi=32768, block=16, quant=False, causal=True, window=4096,
             sinks=4),
        # prompts prefilled under a window with sinks
        dict(name="window prefill, GQA, 2 x 6000", op=w, kind="gqa", heads=64, seqs=2, q_lo=5003,
             q_hi=6000, kv_lo=5003, kv_hi=6000, block=64, quant=False, causal=True, window=1024,
             sinks=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "attention", "attention", "window", "window"])
    kind = rng.choice(sorted(KINDS))
    if op in ("quantize", "dequantize"):
        layers, rows = _log(rng, 1, 61), _log(rng, 1, 16384)
        cd, h, d, _ = KINDS[kind]
        while layers * rows * (cd + h * d) > 16 * 9001 * 8192:
            layers, rows = max(1, layers // 2), max(1, rows * 2 // 3)
        return dict(op=op, kind=kind, layers=layers, rows=rows,
                    slots=64 * (rows // 64 + 1 + _log(rng, 1, 40)))
    heads = {"mla": rng.choice([16, 32, 64, 128]), "gqa": rng.choice([8, 32, 40, 64]),
             "gqa4": rng.choice([4, 16, 28]), "mha": 32}[kind]
    seqs, q, kv = _log(rng, 1, 64), _log(rng, 1, 4096), _log(rng, 16, 32768)
    if rng.random() < 0.4:
        q = 1
    kv = max(kv, q)
    cd, h, d, _ = KINDS[kind]
    wide = 4 if kind == "mla" else 1
    while seqs > 1 and (seqs * heads * q * kv * wide > 32 * 4096 * 16384 // 2 or
                        seqs * kv * h * d > 1 << 29):
        seqs = seqs * 2 // 3
    while seqs * heads * q * kv * wide > 32 * 4096 * 16384 // 2:
        q = max(1, q * 2 // 3)
    win = op == "window"
    return dict(op=op, kind=kind, heads=heads, seqs=seqs, q_lo=max(1, q // 2), q_hi=q,
                kv_lo=max(q, kv // 3), kv_hi=kv, block=rng.choice([16, 64]),
                quant=rng.random() < 0.4, causal=win or rng.random() < 0.8,
                window=_log(rng, 64, 8192) if win else 0,
                sinks=rng.choice([0, 1, 4, 67]) if win else 0)


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["seqs"]
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    kv = [max(a, r.randint(case["kv_lo"], case["kv_hi"])) for a in q]
    q[-1], kv[-1] = case["q_hi"], case["kv_hi"]
    return q, kv


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
    cd, h, d, _ = KINDS[case["kind"]]
    kept = 2 * d if case["kind"] == "mla" else h * d + 4 * (h * d // GROUP)
    row_q = cd + 4 * (cd // GROUP) + kept
    row_b = 2 * (cd + h * d)
    if case["op"] in ("quantize", "dequantize"):
        n = case["layers"] * case["rows"]
        return {"bytes": n * (row_q + row_b) + 4 * case["rows"], "flops": 2 * n * (cd + h * d)}
    dk, dv = (cd + d, cd) if case["kind"] == "mla" else (d, d)
    q, kv = _lengths(case)
    seen = [_pairs(case, a, b) for a, b in zip(q, kv)]
    tokens = sum(q)
    io = tokens * case["heads"] * (2 * (dk + dv) + 4)
    return {"bytes": io + sum(s for _, s in seen) * (row_q if case["quant"] else row_b),
            "flops": 2 * (dk + dv) * case["heads"] * sum(p for p, _ in seen)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(g, shape):
    """Cache rows: unit normal, every 16th channel six times as large, as the
    keys and latents of trained models have a few channels that stand out."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x[..., ::16] *= 6.0
    return x.to(torch.bfloat16)


def _pool(g, kind, layers, slots):
    """bf16 (verbatim, rotary) views in the library's layout."""
    cd, h, d, _ = KINDS[kind]
    if kind == "mla":
        row = torch.empty(layers, slots, cd + d, device="cuda", dtype=torch.bfloat16)
        for l in range(layers):
            row[l] = _rows(g, (slots, cd + d))
        return row[..., :cd], row[..., cd:]
    copy = torch.empty(layers, slots, cd, device="cuda", dtype=torch.bfloat16)
    rot = torch.empty(layers, slots, h * d, device="cuda", dtype=torch.bfloat16)
    for l in range(layers):
        copy[l], rot[l] = _rows(g, (slots, cd)), _rows(g, (slots, h * d))
    return copy, rot


def _quant_pool(kind, layers, slots):
    """Empty quantised pool: e4m3 values and fp32 scales; MLA keeps k_pe in bf16."""
    cd, h, d, _ = KINDS[kind]
    f8, bf, f4 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
    z = lambda w, t: torch.zeros(layers, slots, w, device="cuda", dtype=t)  # noqa: E731
    p = {"copy": z(cd, f8), "copy_scale": z(cd // GROUP, f4)}
    if kind == "mla":
        return {**p, "rot": z(d, bf), "rot_scale": None}
    return {**p, "rot": z(h * d, f8), "rot_scale": z(h * d // GROUP, f4)}


def _desc(kv, kind, copy, rot, block):
    _, h, _, base = KINDS[kind]
    return kv.pool_desc(copy, rot, block, h, base)


def _qdesc(kv, kind, p, block):
    return kv.quant_pool_desc(p["copy"], p["copy_scale"], p["rot"], p["rot_scale"], block,
                              KINDS[kind][1])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]
    cd, h, d, _ = KINDS[kind]
    s = {"case": case}
    if case["op"] in ("quantize", "dequantize"):
        n = case["rows"]
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:n].int()
        s["rows"] = _pool(g, kind, case["layers"], n)
        s["q"] = _quant_pool(kind, case["layers"], case["slots"])
        if case["op"] == "dequantize":  # the registry that is read holds quantised rows
            for l in range(case["layers"]):
                c, r = _pool(g, kind, 1, case["slots"])
                s["q"]["copy"][l], s["q"]["copy_scale"][l] = _quantize(c[0])
                if kind == "mla":
                    s["q"]["rot"][l] = r[0]
                else:
                    s["q"]["rot"][l], s["q"]["rot_scale"][l] = _quantize(r[0])
        if own:
            import position_independent_mla_gb300 as kv
            s["rd"] = _desc(kv, kind, *s["rows"], 1)
            s["qd"] = _qdesc(kv, kind, s["q"], 64)
            s["ws"] = kv.quant_workspace(s["qd"])
        return s
    ql, kl = _lengths(case)
    b, layers = case["block"], 2
    per = -(-max(kl) // b)
    blocks = case["seqs"] * per + 3
    s["layer"] = 1
    s["table"] = torch.randperm(blocks, generator=g, device="cuda")[: case["seqs"] * per].int()
    s["table"] = s["table"].view(case["seqs"], per)
    off = torch.tensor([0] + ql).cumsum(0)
    s["q_off"], s["kv_len"] = off.int().cuda(), torch.tensor(kl, dtype=torch.int32).cuda()
    n = int(off[-1])
    s["seq"] = torch.repeat_interleave(torch.arange(case["seqs"]), torch.tensor(ql)).cuda()
    s["idx"] = torch.arange(n).cuda() - s["q_off"].long()[s["seq"]]
    s["max_q"], s["max_kv"] = max(ql), max(kl)
    dk, dv = (cd + d, cd) if kind == "mla" else (d, d)
    s["scale"] = 192 ** -0.5 if kind == "mla" else 128 ** -0.5
    s["query"] = torch.randn(n, case["heads"], dk, generator=g, device="cuda").to(torch.bfloat16)
    pool = _pool(g, kind, layers, blocks * b)
    if case["quant"]:
        s["pool"] = dict(zip(("copy", "copy_scale"), _quantize(pool[0])))
        s["pool"]["rot"], s["pool"]["rot_scale"] = ((pool[1].contiguous(), None) if kind == "mla"
                                                    else _quantize(pool[1]))
    else:
        s["pool"] = {"copy": pool[0], "rot": pool[1]}
    s["out"] = torch.empty(n, case["heads"], dv, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.empty(n, case["heads"], device="cuda", dtype=torch.float32)
    if own:
        import position_independent_mla_gb300 as kv
        s["pd"] = (_qdesc(kv, kind, s["pool"], b) if case["quant"]
                   else _desc(kv, kind, s["pool"]["copy"], s["pool"]["rot"], b))
        s["ad"] = kv.attn_desc(s["q_off"], s["kv_len"], s["table"], max_q_len=max(ql),
                               max_kv_len=max(kl), scale=s["scale"], causal=case["causal"],
                               window=case["window"], sinks=case["sinks"])
        s["ws"] = kv.attn_workspace(s["pd"], s["ad"], s["query"])
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def _quantize(x):
    """e4m3 values and scales: 2^e with the smallest e that keeps a group's
    largest finite magnitude at or below 448; values that are not finite are NaN."""
    y = x.float().reshape(*x.shape[:-1], -1, GROUP)
    top = torch.where(torch.isfinite(y), y.abs(), torch.zeros_like(y)).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top == 0, 0, (e - 9 + (m > 0.875)).clamp(min=-120))
    scale = torch.ldexp(torch.ones_like(top), e)
    y = y * torch.ldexp(torch.ones_like(top), -e).unsqueeze(-1)
    y = torch.where(torch.isfinite(y), y, torch.full_like(y, math.nan))
    return y.to(torch.float8_e4m3fn).reshape(x.shape), scale


def _value(x8, scale):
    y = x8.float()
    if scale is None:
        return y
    return (y.reshape(*y.shape[:-1], -1, GROUP) * scale.unsqueeze(-1)).reshape(y.shape)


def _at(t, layer, slots):
    """Rows of a layer at the slots (8-bit values are indexed as bytes)."""
    if t is None:
        return None
    return (t[layer].view(torch.uint8)[slots].view(t.dtype) if t.dtype == torch.float8_e4m3fn
            else t[layer][slots])


def _attend(s):
    case, pool, l = s["case"], s["pool"], s["layer"]
    cd, h, d, _ = KINDS[case["kind"]]
    b, nk, nq = case["block"], s["max_kv"], s["max_q"]
    k = torch.arange(nk, device="cuda")
    slots = s["table"].long()[:, k // b] * b + k % b                       # [S, K]
    copy = _value(_at(pool["copy"], l, slots), _at(pool.get("copy_scale"), l, slots))
    rot = _value(_at(pool["rot"], l, slots), _at(pool.get("rot_scale"), l, slots))
    if case["kind"] == "mla":
        key, val = torch.cat([copy, rot], -1).unsqueeze(2), copy.unsqueeze(2)
    else:
        key, val = rot.unflatten(-1, (h, d)), copy.unflatten(-1, (h, d))   # [S, K, h, d]
    heads = case["heads"]
    q = torch.zeros(case["seqs"], nq, heads, s["query"].shape[-1], device="cuda")
    q[s["seq"], s["idx"]] = s["query"].float()
    q = q.unflatten(2, (h, heads // h)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [S, h, g*nq, d]
    score = (q @ key.permute(0, 2, 3, 1)).mul_(s["scale"])                 # [S, h, g*nq, K]
    score = score.unflatten(2, (heads // h, nq))
    i = torch.arange(nq, device="cuda")
    length = s["kv_len"].long()[:, None, None]
    pos = length - (s["q_off"][1:] - s["q_off"][:-1]).long()[:, None, None] + i[None, :, None]
    see = (k < length).expand(-1, nq, -1)
    if case["causal"]:
        see = see & (k <= pos)
    if case["window"]:
        see = see & ((k > pos - case["window"]) | (k < case["sinks"]))
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1)
    out = p.flatten(2, 3) @ val.permute(0, 2, 1, 3)                        # [S, h, g*nq, dv]
    out = out.unflatten(2, (heads // h, nq)) / total.clamp(min=1e-38).unsqueeze(-1)
    lse = total.log() + top.squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["seq"], s["idx"]]
    return out.to(torch.bfloat16), lse.permute(0, 3, 1, 2).flatten(2, 3)[s["seq"], s["idx"]]


def run(s):
    case = s["case"]
    mla = case["kind"] == "mla"
    if case["op"] == "quantize":
        q = s["q"]
        if own:
            import position_independent_mla_gb300 as kv
            kv.kv_quantize(s["rd"], None, s["qd"], 0, case["rows"], s["slots"], s["ws"])
        else:
            copy, rot, at = *s["rows"], s["slots"].long()
            x8, scale = _quantize(copy)
            q["copy"].view(torch.uint8)[:, at] = x8.view(torch.uint8)
            q["copy_scale"][:, at] = scale
            if mla:
                q["rot"][:, at] = rot
            else:
                x8, scale = _quantize(rot)
                q["rot"].view(torch.uint8)[:, at] = x8.view(torch.uint8)
                q["rot_scale"][:, at] = scale
        return q
    if case["op"] == "dequantize":
        if own:
            import position_independent_mla_gb300 as kv
            kv.kv_dequantize(s["qd"], 0, s["slots"], s["rd"], case["rows"], None, s["ws"])
            return s["rows"]
        q, at = s["q"], (slice(None), s["slots"].long())
        rot = (q["rot"][at] if mla
               else _value(q["rot"].view(torch.uint8)[at].view(torch.float8_e4m3fn),
                           q["rot_scale"][at]).to(torch.bfloat16))
        copy = _value(q["copy"].view(torch.uint8)[at].view(torch.float8_e4m3fn),
                      q["copy_scale"][at])
        return copy.to(torch.bfloat16), rot
    if own:
        import position_independent_mla_gb300 as kv
        kv.kv_attention(s["pd"], s["layer"], s["ad"], s["query"], s["out"], s["lse"], s["ws"])
        return s["out"], s["lse"]
    return _attend(s)


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_e4m3(x):
    """Values and scales of one layer's rows, the rounding to four significant
    bits (steps of 2^-9 below 2^-6) written out in double precision."""
    v = x.double().reshape(x.shape[0], -1, GROUP)
    top = torch.nan_to_num(v.abs(), nan=0.0, posinf=0.0).amax(-1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0) - 1e-12).clamp(min=-120)
    v = v * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).reshape(x.shape), torch.exp2(e).float().double()


def exact(case, seed):
    s = prepare(case, seed)
    kind, mla = case["kind"], case["kind"] == "mla"
    cd, h, d, _ = KINDS[kind]
    if case["op"] == "quantize":
        out = {k: None if t is None else torch.zeros(t.shape, device="cuda", dtype=torch.float32)
               for k, t in s["q"].items()}
        at = s["slots"].long()
        for l in range(case["layers"]):
            for name, t in zip(("copy", "rot"), s["rows"]):
                if mla and name == "rot":
                    out[name][l, at] = t[l].float()
                    continue
                v, e = _exact_e4m3(t[l])
                out[name][l, at], out[name + "_scale"][l, at] = v.float(), e.float()
        return {k: v for k, v in out.items()}
    if case["op"] == "dequantize":
        at = s["slots"].long()
        got = []
        for name, w in (("copy", cd), ("rot", h * d)):
            v = torch.empty(case["layers"], case["rows"], w, device="cuda", dtype=torch.float32)
            for l in range(case["layers"]):
                x = s["q"][name][l].to(torch.float32)[at].double()
                if s["q"][name + "_scale"] is not None:
                    x = x * s["q"][name + "_scale"][l][at].double().repeat_interleave(GROUP, -1)
                v[l] = x.float()
            got.append(v)
        return tuple(got)
    ql, kl = _lengths(case)
    dv, heads, b, l = (cd if mla else d), case["heads"], case["block"], s["layer"]
    out = torch.empty(sum(ql), heads, dv, device="cuda", dtype=torch.float64)
    lse = torch.empty(sum(ql), heads, device="cuda", dtype=torch.float64)
    at = 0
    for q, nq, nk in zip(range(case["seqs"]), ql, kl):
        pos = torch.arange(nk, device="cuda")
        slot = s["table"][q].long()[pos // b] * b + pos % b
        part = {}
        for name in ("copy", "rot"):
            x = s["pool"][name][l].to(torch.float32)[slot].double()
            sc = s["pool"].get(name + "_scale")
            part[name] = x if sc is None else x * sc[l][slot].double().repeat_interleave(GROUP, -1)
        mine = nk - nq + torch.arange(nq, device="cuda")
        far = mine[:, None] - pos[None, :]
        ok = torch.ones_like(far, dtype=torch.bool) if not case["causal"] else far >= 0
        if case["window"]:
            ok = ok & ((far < case["window"]) | (pos < case["sinks"])[None, :])
        bias = torch.where(ok, 0.0, -math.inf).double()
        for head in range(heads):
            j = head // (heads // h)
            key = torch.cat([part["copy"], part["rot"]], 1) if mla else part["rot"][:, j * d:j * d + d]
            val = part["copy"] if mla else part["copy"][:, j * d:j * d + d]
            z = s["query"][at:at + nq, head].double() @ key.T * s["scale"] + bias
            n = torch.logsumexp(z, -1)
            lse[at:at + nq, head] = n
            n = torch.where(n == -math.inf, 0.0, n)
            out[at:at + nq, head] = torch.exp(z - n[:, None]) @ val
        at += nq
    return out, lse
