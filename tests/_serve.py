"""Inputs and 64-bit references of the quantised-row and attention tests."""
from __future__ import annotations

import math
from types import SimpleNamespace

import torch

import position_independent_mla_gb300 as kv

SHAPES = {  # copy_dim, rot_heads, rot_head_dim, rope_base
    "mla": (512, 1, 64, 10000.0),
    "gqa": (1024, 8, 128, 500000.0),
    "gqa4": (512, 4, 128, 1000000.0),
    "mha": (4096, 32, 128, 10000.0),
}


def ref_quantize(x):
    """(values, scales) in 64 bits of rows x [..., width]: the e4m3 rounding
    written out (steps of a quarter of 2^-1 of the leading bit, 2^-9 at least)."""
    v = x.double().unflatten(-1, (-1, 128))
    top = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(-1)
    e = torch.zeros_like(top)
    for i in range(top.numel()):
        a, k = float(top.view(-1)[i]), -120
        if a > 0:
            while a > 448.0 * 2.0 ** k:
                k += 1
            e.view(-1)[i] = k
    v = v * torch.exp2(-e).unsqueeze(-1)
    v = torch.where(torch.isfinite(v), v, torch.full_like(v, math.nan))
    lead = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(lead - 3)
    return (torch.round(v / step) * step).flatten(-2), torch.exp2(e)


def bf16_rows(g, *shape, outliers=True):
    x = torch.randn(shape, generator=g, dtype=torch.float32)
    if outliers:
        x[..., ::16] *= 6.0
    return x.to(torch.bfloat16)


def empty_quant(kind, layers, slots, block, pad=0):
    """An empty quantised pool; ``pad`` extra columns make the slot strides odd
    multiples of the alignment."""
    cd, h, d, _ = SHAPES[kind]
    z = lambda w, t, p: torch.zeros(layers, slots, w + p, dtype=t, device="cuda")[..., :w]  # noqa: E731
    f8, f4 = torch.float8_e4m3fn, torch.float32
    copy, cs = z(cd, f8, 16 * pad), z(cd // 128, f4, pad)
    rot = z(d, torch.bfloat16, 8 * pad) if kind == "mla" else z(h * d, f8, 16 * pad)
    rs = None if kind == "mla" else z(h, f4, pad)
    return SimpleNamespace(kind=kind, copy=copy, copy_scale=cs, rot=rot, rot_scale=rs,
                           desc=kv.quant_pool_desc(copy, cs, rot, rs, block, h))


def value64(x8, scale):
    v = x8.float().double()
    return v if scale is None else (v.unflatten(-1, (-1, 128)) * scale.double().unsqueeze(-1)).flatten(-2)


class Batch:
    """A paged pool and a ragged batch over it; ``lens`` = [(new, cached), ...]."""

    def __init__(self, kind, lens, heads, seed=1, block=64, quant=False, q_scale=1.0,
                 causal=True, window=0, sinks=0, strided=False, table_pad=2):
        g = torch.Generator().manual_seed(seed)
        cd, h, d, base = SHAPES[kind]
        self.kind, self.lens, self.heads, self.block, self.quant = kind, lens, heads, block, quant
        self.mla, self.h, self.d = kind == "mla", h, d
        self.causal, self.window, self.sinks = causal, window, sinks
        per = max(1, -(-max(b for _, b in lens) // block)) + table_pad
        blocks = len(lens) * per + 2
        self.layers, self.layer, slots = 2, 1, blocks * block
        self.table = torch.randperm(blocks, generator=g)[: len(lens) * per].int().view(len(lens), per)
        copy = bf16_rows(g, self.layers, slots, cd)
        rot = bf16_rows(g, self.layers, slots, h * d)
        if quant:
            self.pool = empty_quant(kind, self.layers, slots, block, pad=1 if strided else 0)
            src = kv.pool_desc(copy.cuda(), rot.cuda(), 1, h, base)
            ws = kv.quant_workspace(self.pool.desc)
            kv.kv_quantize(src, None, self.pool.desc, 0, slots,
                           torch.arange(slots, dtype=torch.int32, device="cuda"), ws)
            assert kv.kv_get_device_status(ws) == kv.KV_OK
            self.desc = self.pool.desc
        elif self.mla:
            row = torch.cat([copy, rot], -1).cuda()
            self.pool = SimpleNamespace(copy=row[..., :cd], rot=row[..., cd:], copy_scale=None,
                                        rot_scale=None)
            self.desc = kv.pool_desc(self.pool.copy, self.pool.rot, block, h, base)
        else:
            w = cd + (64 if strided else 0)
            both = torch.zeros(2, self.layers, slots, w, dtype=torch.bfloat16, device="cuda")
            both[0, ..., :cd], both[1, ..., :cd] = copy.cuda(), rot.cuda()
            self.pool = SimpleNamespace(copy=both[0, ..., :cd], rot=both[1, ..., :cd],
                                        copy_scale=None, rot_scale=None)
            self.desc = kv.pool_desc(self.pool.copy, self.pool.rot, block, h, base)
        n = sum(a for a, _ in lens)
        self.n, self.dk, self.dv = n, 576 if self.mla else 128, 512 if self.mla else 128
        q = (torch.randn(n, heads, self.dk, generator=g) * q_scale).to(torch.bfloat16).cuda()
        if strided:  # heads outside tokens, rows wider than the head
            wide = torch.zeros(heads, n, self.dk + 8, dtype=torch.bfloat16, device="cuda")
            self.q = wide.transpose(0, 1)[..., : self.dk]
            self.q.copy_(q)
            self.out = torch.full((heads, n, self.dv + 24), 7.0, dtype=torch.bfloat16,
                                  device="cuda").transpose(0, 1)[..., : self.dv]
        else:
            self.q = q
            self.out = torch.full((n, heads, self.dv), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, heads), 7.0, device="cuda")
        off = torch.tensor([0] + [a for a, _ in lens]).cumsum(0).int()
        self.scale = 1.0 / math.sqrt(192 if self.mla else 128)
        self.attn = kv.attn_desc(off.cuda(), torch.tensor([b for _, b in lens], dtype=torch.int32).cuda(),
                                 self.table.cuda(), max(a for a, _ in lens),
                                 max(b for _, b in lens), self.scale, causal, window, sinks)
        self.ws = kv.attn_workspace(self.desc, self.attn, self.q)

    def slots(self, s):
        k = torch.arange(self.lens[s][1])
        return self.table[s].long()[k // self.block] * self.block + k % self.block

    def run(self, status=kv.KV_OK):
        kv.kv_attention(self.desc, self.layer, self.attn, self.q, self.out, self.lse, self.ws)
        assert kv.kv_get_device_status(self.ws) == status
        return self.out, self.lse

    def visible(self, s):
        n, m = self.lens[s]
        p, k = m - n + torch.arange(n)[:, None], torch.arange(m)[None, :]
        ok = torch.ones(n, m, dtype=torch.bool)
        if self.causal:
            ok &= k <= p
        if self.window:
            ok &= (k > p - self.window) | (k < self.sinks)
        return ok

    def reference(self):
        """Per sequence (out, lse, bound of |out|, bound of |lse|) in 64 bits.

        Bounds, derived: bf16 has 8 significant bits (its spacing in [1, 2) is
        2^-7), so rounding to nearest is off by at most 2^-8 of the value.  The
        weights are rounded once (2^-8 of each, so 2^-8 of A = sum p|v|) and out
        once (2^-8 |out|).  A score is an fp32 sum of
        at most 576 exact products: its error is below 2^-20 of scale * sum|q||k|
        = B, and shifts every weight and lse by no more than that; exp2, the
        running sums and their rescaling add less than 2^-16 of a weight."""
        got = []
        at = 0
        for s, (n, m) in enumerate(self.lens):
            slots = self.slots(s).cuda()
            part = []
            for name in ("copy", "rot"):
                x = getattr(self.pool, name)[self.layer].float()[slots]
                sc = getattr(self.pool, name + "_scale")
                part.append(value64(x, None if sc is None else sc[self.layer][slots]))
            copy, rot = part
            if self.mla:
                key, val = torch.cat([copy, rot], -1)[None], copy[None]
            else:
                key = rot.unflatten(-1, (self.h, 128)).transpose(0, 1)
                val = copy.unflatten(-1, (self.h, 128)).transpose(0, 1)
            g = self.heads // self.h
            key, val = key.repeat_interleave(g, 0), val.repeat_interleave(g, 0)
            q = self.q[at:at + n].double().transpose(0, 1)
            ok = self.visible(s).cuda()
            z = (q @ key.transpose(1, 2)) * self.scale
            z = torch.where(ok, z, torch.full_like(z, -math.inf))
            mag = (q.abs() @ key.abs().nan_to_num().transpose(1, 2)) * self.scale
            mag = torch.where(ok, mag, torch.zeros_like(mag)).amax(-1) if m else torch.zeros(self.heads, n, device="cuda").double()
            if m:
                lse = torch.logsumexp(z, -1)
                p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
                # a key that is not seen has no part, whatever it holds
                bad = ~torch.isfinite(val)
                out = p @ torch.where(bad, torch.zeros_like(val), val)
                if bad.any():
                    seen = (p * ok) @ bad.double()
                    out = torch.where(seen > 0, torch.full_like(out, math.nan), out)
                a = p @ val.abs().nan_to_num()
            else:
                lse = torch.full((self.heads, n), -math.inf, device="cuda").double()
                out = torch.zeros(self.heads, n, self.dv, device="cuda").double()
                a = out.clone()
            b = mag * 2.0 ** -20
            tol_o = 2.0 ** -8 * out.abs() + a * (2.0 ** -8 + 2.0 ** -16 + 2 * b)[..., None]
            tol_l = b + 2.0 ** -16
            got.append(tuple(t.transpose(0, 1) for t in (out, lse, tol_o, tol_l)))
            at += n
        return [torch.cat(t) for t in zip(*got)]

    def check(self):
        out, lse = self.run()
        want, wl, to, tl = self.reference()
        o = out.double()
        assert torch.equal(torch.isnan(o), torch.isnan(want)), "NaN pattern of out"
        fin = ~torch.isnan(want)
        err = (o - want).abs()[fin]
        bad = err > to[fin]
        assert not bad.any(), f"out: {int(bad.sum())} of {bad.numel()} beyond bound, max {float(err.max()):.3g}"
        nan = torch.isnan(wl)
        assert torch.equal(torch.isnan(lse), nan), "NaN pattern of lse"
        inf = torch.isinf(wl)
        assert torch.equal(lse[inf].double(), wl[inf]), "lse of empty rows"
        ok = ~(nan | inf)
        assert not ((lse.double() - wl).abs()[ok] > tl[ok]).any(), "lse beyond bound"
        return out, lse
