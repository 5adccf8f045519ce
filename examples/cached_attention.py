"""A question over cached documents: the serving calls together.

A registry keeps canonical chunks (prefilled from position 0) as e4m3 rows.  A
request reuses them: their rows are read back (kv_dequantize), moved behind
the request's prompt with their keys turned to the new positions (kv_relocate), and the
question's tokens attend to the whole context as one chunk, then token by token as
the answer grows (kv_attention), in full and with a sliding window behind the first
tokens.  Everything is compared with dense attention in 64 bits over rows that were
never quantised, keys rotated straight to their positions: what differs is the
cache's rounding to e4m3 (3.6 % of a value in the mean square, at most).

    python examples/cached_attention.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import position_independent_mla_gb300 as kv  # noqa: E402

BASE, BLOCK, HEADS = 10000.0, 64, 16
LATENT, ROPE = 512, 64


def rotate(x, pos):
    """Rotate-half RoPE of rows x [n, 64] at positions pos [n], in 64 bits."""
    j = torch.arange(ROPE // 2, dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] * BASE ** (-2.0 * j / ROPE)
    a, b = x.double().chunk(2, -1)
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)


def dense(q, rows, scale, window, sinks):
    """Causal attention of the last len(q) rows' queries, in 64 bits."""
    n, m = q.shape[0], rows.shape[0]
    z = torch.einsum("thd,kd->htk", q.double(), rows.double()) * scale
    key = torch.arange(m, device=q.device)[None]
    own = m - n + torch.arange(n, device=q.device)[:, None]
    seen = key <= own
    if window:
        seen &= (key > own - window) | (key < sinks)
    p = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
    return torch.einsum("htk,kd->thd", p, rows.double()[:, :LATENT])


def run(chunk_lens=(300, 170), prompt=45, question=23, answer=4, seed=0):
    """Returns the root mean square error of the question's and the answer tokens'
    attention, relative to the outputs' root mean square: without a window, then with."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    layer, layers = 1, 2
    total = prompt + sum(chunk_lens) + question + answer

    # the registry: canonical chunks, keys at positions 0, 1, ..., written as e4m3
    slots = sum(chunk_lens)
    reg_slots = -(-slots // BLOCK) * BLOCK
    latent = torch.zeros(layers, reg_slots, LATENT, dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.zeros(layers, reg_slots, LATENT // 128, device=dev)
    k_pe = torch.zeros(layers, reg_slots, ROPE, dtype=torch.bfloat16, device=dev)
    registry = kv.quant_pool_desc(latent, scales, k_pe, None, BLOCK, 1)
    base_latent, base_key = draw(layers, slots, LATENT), draw(layers, slots, ROPE)
    start = torch.cat([torch.arange(n, device=dev) for n in chunk_lens])
    keys = torch.stack([rotate(base_key[l], start) for l in range(layers)]).bfloat16()
    fresh = kv.pool_desc(base_latent.bfloat16(), keys, 1, 1, BASE)
    at = torch.randperm(reg_slots, generator=g, device=dev)[:slots].int()
    qws = kv.quant_workspace(registry)
    kv.kv_quantize(fresh, None, registry, 0, slots, at, qws)

    # a hit: rows back in bf16, then into the request's pool behind its prompt
    stage = torch.empty(layers, reg_slots, LATENT + ROPE, dtype=torch.bfloat16, device=dev)
    staged = kv.pool_desc(stage[..., :LATENT], stage[..., LATENT:], BLOCK, 1, BASE)
    kv.kv_dequantize(registry, 0, at, staged, slots, None, qws)
    blocks = -(-total // BLOCK)
    pool = torch.zeros(layers, (blocks + 2) * BLOCK, LATENT + ROPE, dtype=torch.bfloat16, device=dev)
    desc = kv.pool_desc(pool[..., :LATENT], pool[..., LATENT:], BLOCK, 1, BASE)
    table = torch.randperm(blocks + 2, generator=g, device=dev)[:blocks].int()[None].contiguous()
    offsets = [sum(chunk_lens[:i]) for i in range(len(chunk_lens) + 1)]
    targets = [prompt + o for o in offsets[:-1]]
    ws = kv.workspace(desc, slots, len(chunk_lens))
    kv.kv_relocate(staged, desc, len(chunk_lens), slots, i32(*offsets),
                   torch.arange(slots, dtype=torch.int32, device=dev),
                   i32(*[0 for _ in chunk_lens]), i32(*targets),
                   i32(*targets), table, 1, blocks, None, ws)

    # the prompt's, the question's and the answer's own rows, at their positions
    pos = torch.arange(total, device=dev)
    place = table[0].long()[pos // BLOCK] * BLOCK + pos % BLOCK
    own = torch.ones(total, dtype=torch.bool, device=dev)
    own[prompt:prompt + slots] = False
    own_latent, own_key = draw(int(own.sum()), LATENT), draw(int(own.sum()), ROPE)
    pool[layer, place[own]] = torch.cat([own_latent, rotate(own_key, pos[own]).float()], -1).bfloat16()

    # what all rows would be without a cache
    rows = torch.empty(total, LATENT + ROPE, dtype=torch.float64, device=dev)
    rows[own] = torch.cat([own_latent.double(), rotate(own_key, pos[own])], -1)
    rows[~own] = torch.cat([base_latent[layer].double(), rotate(base_key[layer], pos[~own])], -1)

    scale = 192 ** -0.5
    q = draw(question + answer, HEADS, LATENT + ROPE).bfloat16()
    errors = []

    def attend(n, length, window=0, sinks=0):
        query = q[length - n - (total - question - answer):][:n]
        batch = kv.attn_desc(i32(0, n), i32(length), table, n, length, scale, True, window, sinks)
        out = torch.empty(n, HEADS, LATENT, dtype=torch.bfloat16, device=dev)
        aws = kv.attn_workspace(desc, batch, query)
        kv.kv_attention(desc, layer, batch, query, out, None, aws)
        assert kv.kv_get_device_status(aws) == kv.KV_OK
        want = dense(query, rows[:length], scale, window, sinks)
        errors.append(float(((out.double() - want).square().mean() / want.square().mean()).sqrt()))

    for window, sinks in ((0, 0), (100, 4)):
        attend(question, total - answer, window, sinks)
        for i in range(answer):
            attend(1, total - answer + 1 + i, window, sinks)
    assert kv.kv_get_device_status(qws) == kv.KV_OK and kv.kv_get_device_status(ws) == kv.KV_OK
    return errors


if __name__ == "__main__":
    errs = run()
    half = len(errs) // 2
    for name, e in (("full", errs[:half]), ("window 100 + 4 sinks", errs[half:])):
        print("%s: rms error / rms, question %.4f, answer tokens %s"
              % (name, e[0], ", ".join("%.4f" % x for x in e[1:])))
