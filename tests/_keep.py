"""Inputs and 64-bit references of the tests of drafted trees and bounded caches."""
from __future__ import annotations

import math

import torch

import position_independent_mla_gb300 as kv
from _serve import Batch, value64


class Tree(Batch):
    """A batch whose new tokens are trees; ``masks[s][i]``: bits of the new tokens that query i
    of sequence s sees (default: random trees)."""

    def __init__(self, kind, lens, heads, masks=None, extra_words=0, **k):
        super().__init__(kind, lens, heads, causal=False, **k)
        g = torch.Generator().manual_seed(k.get("seed", 1) + 77)
        if masks is None:
            masks = []
            for n, _ in lens:
                sees = []
                for j in range(n):
                    up = int(torch.randint(0, max(1, j), (1,), generator=g)) if j else -1
                    sees.append((sees[up] if j else 0) | 1 << j)
                masks.append(sees)
        self.masks = masks
        words = max(1, -(-max(n for n, _ in lens) // 32)) + extra_words
        rows = [[(x >> 32 * w) & 0xFFFFFFFF for w in range(words)] for s in masks for x in s]
        bits = torch.tensor(rows, dtype=torch.int64).reshape(-1, words)
        self.mask = (bits - ((bits >> 31) << 32)).to(torch.int32).cuda()
        self.ws = kv.tree_workspace(self.desc, self.attn, self.q)

    def visible(self, s):
        n, m = self.lens[s]
        ok = torch.zeros(n, m, dtype=torch.bool)
        ok[:, :max(0, m - n)] = True
        for i in range(n):
            for j in range(n):
                if m - n + j >= 0 and (self.masks[s][i] >> j) & 1:
                    ok[i, m - n + j] = True
        return ok

    def run(self, status=kv.KV_OK):
        kv.kv_tree_attention(self.desc, self.layer, self.attn, self.mask, self.q, self.out,
                             self.lse, self.ws)
        assert kv.kv_get_device_status(self.ws) == status
        return self.out, self.lse


class Sums(Batch):
    """A batch, its queries' lse and earlier weights."""

    def __init__(self, kind, lens, heads, keep=1.0, pad=3, **k):
        super().__init__(kind, lens, heads, **k)
        self.keep = keep
        most = max(1, max(m for _, m in lens))
        g = torch.Generator().manual_seed(k.get("seed", 1) + 5)
        self.weights = torch.rand(len(lens), most + pad, generator=g).cuda()
        self.lse = self.scores_lse().float().contiguous()
        self.wws = kv.weights_workspace(self.desc, self.attn, self.q)

    def parts(self, s):
        """(scores [heads, n, m], their magnitudes, visible) of sequence s in 64 bits."""
        n, m = self.lens[s]
        at = sum(a for a, _ in self.lens[:s])
        slots = self.slots(s).cuda()
        part = []
        for name in ("copy", "rot"):
            x = getattr(self.pool, name)[self.layer].float()[slots]
            sc = getattr(self.pool, name + "_scale")
            part.append(value64(x, None if sc is None else sc[self.layer][slots]))
        key = (torch.cat(part, -1)[None] if self.mla
               else part[1].unflatten(-1, (self.h, 128)).transpose(0, 1))
        key = key.repeat_interleave(self.heads // self.h, 0)
        q = self.q[at:at + n].double().transpose(0, 1)
        return (q @ key.transpose(1, 2) * self.scale,
                q.abs() @ key.abs().transpose(1, 2) * self.scale, self.visible(s).cuda())

    def scores_lse(self):
        rows = []
        for s, (n, m) in enumerate(self.lens):
            z, _, ok = self.parts(s)
            z = torch.where(ok, torch.nan_to_num(z, nan=0.0), torch.full_like(z, -math.inf))
            rows.append(torch.logsumexp(z, -1).T if m else
                        torch.full((n, self.heads), -math.inf, device="cuda").double())
        return torch.cat(rows)

    def run(self, status=kv.KV_OK):
        kv.kv_attention_weights(self.desc, self.layer, self.attn, self.q, self.lse, self.weights,
                                self.keep, self.wws)
        assert kv.kv_get_device_status(self.wws) == status
        return self.weights

    def run_attention(self):
        """(out, lse) of kv_attention over the same keys."""
        return Batch.run(self)

    def check(self):
        """Bounds, derived: a score is an fp32 sum of at most 576 exact products, off by less
        than 2^-20 of B = scale * sum|q||k|; the exponent is formed with a rounding each of
        scale * log2 e, of lse * log2 e (two) and of their difference, together below 2^-22 of
        |S| + |lse|; exp2 is off by less than 2^-21 of itself.  So a term is off by its value
        times (e^d - 1), d = 2^-20 B + 2^-22 (|S| + |lse|) + 2^-21.  All terms are positive: a sum
        over chains of c additions is off by c 2^-24 of itself, c below 200 + steps (a step adds a
        row tile of a head).  Terms below 2^-126 may be lost.  keep * weights adds a rounding of
        the result."""
        old = self.weights.clone()
        got = self.run().double()
        at = 0
        for s, (n, m) in enumerate(self.lens):
            assert torch.equal(self.weights[s, m:], old[s, m:]), "entries behind the last key"
            z, mag, ok = self.parts(s)
            lse = self.lse[at:at + n].double().T[:, :, None]
            at += n
            e = torch.where(ok & (lse != -math.inf), torch.exp(z - lse), torch.zeros_like(z))
            d = 2.0 ** -20 * mag + 2.0 ** -22 * (z.abs() + lse.abs().nan_to_num(posinf=0.0)) + 2.0 ** -21
            d = torch.where(e == 0, torch.zeros_like(d), d)
            new = e.sum((0, 1))
            tol = (e * torch.expm1(d)).sum((0, 1))
            steps = self.h * (n // max(1, 128 // (self.heads // self.h)) + 1)
            want = self.keep * old[s, :m].double() + new if self.keep else new
            tol = tol + (200 + steps) * 2.0 ** -24 * want.abs() + n * self.heads * 2.0 ** -126
            w = got[s, :m]
            assert torch.equal(torch.isnan(w), torch.isnan(want)), "NaN pattern"
            bad = ((w - want).abs() > tol) & ~torch.isnan(want)
            assert not bad.any(), (s, int(bad.sum()), float(((w - want).abs() / tol).nan_to_num().max()))
        return got


def ref_select(weights, kv_len, budget, sinks, recent):
    """Positions that stay, ascending, of each sequence."""
    got = []
    for w, n, b in zip(weights.tolist(), kv_len, budget):
        w = w[:n]
        fixed = [i for i in range(n) if i < sinks or i >= n - recent]
        rest = [i for i in range(n) if sinks <= i < n - recent]
        rest.sort(key=lambda i: (0, -w[i], i) if w[i] == w[i] else (1, 0.0, i))
        got.append(sorted((fixed + rest)[:b]))
    return got
