"""Argument checks of the calls for drafted trees and bounded caches (no GPU: every call
here is refused before anything is enqueued)."""
import ctypes as C

import pytest
import torch

import position_independent_mla_gb300 as kv
from position_independent_mla_gb300 import build as kbuild
from test_serve_abi_cpu import A, _attn, _pool, _quant

INVALID, UNSUPPORTED, WORKSPACE = kv.KV_ERR_INVALID_ARG, kv.KV_ERR_UNSUPPORTED, kv.KV_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kv.load()


def _mla_quant(**k):
    return _quant(copy_dim=512, copy_slot_stride=512, copy_scale_slot_stride=4, rot_heads=1,
                  rot_head_dim=64, rot_slot_stride=64, rot_scale=None, **k)


def _f(lib, name, pool):
    return getattr(lib, name + ("_quant" if isinstance(pool, kv.kv_quant_pool_desc) else ""))


def _tree(lib, pool=None, layer=0, attn=None, mask=A, ms=1, n=8, heads=32, q=A, qs=(4096, 128),
          out=A, os=(4096, 128), lse=A, ws=A, size=1 << 30):
    pool = pool or _pool()
    return _f(lib, "kv_tree_attention", pool)(
        C.byref(pool), layer, C.byref(attn or _attn()), mask, ms, n, heads, q, *qs, out, *os, lse,
        ws, size, None)


@pytest.mark.parametrize("bad", [
    dict(mask=None), dict(mask=A + 2), dict(ms=0), dict(attn=_attn(max_q_len=33)), dict(layer=2),
    dict(q=None), dict(out=A + 8), dict(heads=33), dict(pool=_quant(rot_base=A + 8)),
    dict(attn=_attn(window=5, causal=0)), dict(attn=_attn(scale=NAN)),
], ids=str)
def test_tree_refuses(lib, bad):
    assert _tree(lib, **bad) == INVALID


def test_tree_refuses_windows_shapes_and_workspaces(lib):
    assert _tree(lib, attn=_attn(window=8)) == UNSUPPORTED
    assert _tree(lib, pool=_pool(rot_heads=2, copy_dim=256)) == UNSUPPORTED
    assert _tree(lib, heads=8 * 129, qs=(8 * 129 * 128, 128)) == UNSUPPORTED
    for w in (dict(ws=None), dict(ws=A + 16), dict(size=256)):
        assert _tree(lib, **w) == WORKSPACE
    p = _pool()
    f = lib.kv_tree_attention_workspace_size
    assert f(C.byref(p), C.byref(_attn(window=8)), 8, 32) == 0
    assert f(C.byref(p), C.byref(_attn()), 8, 32) > 256


def _weights(lib, pool=None, layer=0, attn=None, n=8, heads=32, q=A, qs=(4096, 128), lse=A, w=A,
             stride=100, keep=1.0, ws=A, size=1 << 30):
    pool = pool or _pool()
    return _f(lib, "kv_attention_weights", pool)(
        C.byref(pool), layer, C.byref(attn or _attn()), n, heads, q, *qs, lse, w, stride, keep, ws,
        size, None)


@pytest.mark.parametrize("bad", [
    dict(layer=-1), dict(n=9), dict(heads=0), dict(q=None), dict(q=A + 8), dict(qs=(4096, 4)),
    dict(lse=None), dict(lse=A + 2), dict(w=None), dict(w=A + 1), dict(stride=99), dict(keep=-0.5),
    dict(keep=NAN), dict(keep=INF), dict(attn=_attn(d_q_off=None)), dict(attn=_attn(d_kv_len=None)),
    dict(attn=_attn(d_block_tables=A + 2)), dict(attn=_attn(max_blocks=0)),
    dict(pool=_quant(copy_scale=None)), dict(attn=_attn(window=3, causal=0)),
], ids=str)
def test_weights_refuse(lib, bad):
    assert _weights(lib, **bad) == INVALID


def test_weights_refuse_shapes_and_workspaces(lib):
    assert _weights(lib, pool=_pool(rot_heads=2, copy_dim=256)) == UNSUPPORTED
    assert _weights(lib, heads=8 * 129, qs=(8 * 129 * 128, 128)) == UNSUPPORTED
    for w in (dict(ws=None), dict(ws=A + 16), dict(size=256)):
        assert _weights(lib, **w) == WORKSPACE


def _select(lib, n=2, w=A, ws_=100, kl=A, mk=100, b=A, sinks=0, recent=0, keep=A, ks=50, most=50,
            count=A, kept=A, kst=50, ws=A, size=1 << 20):
    return lib.kv_evict_select(n, w, ws_, kl, mk, b, sinks, recent, keep, ks, most, count, kept,
                               kst, ws, size, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(w=None), dict(w=A + 2), dict(ws_=99), dict(kl=None), dict(kl=A + 1),
    dict(mk=-1), dict(mk=(1 << 30) + 1, ws_=1 << 31), dict(b=None), dict(sinks=-1), dict(recent=-1),
    dict(keep=None), dict(ks=49), dict(most=-1), dict(count=None), dict(count=A + 2), dict(kept=A + 2),
    dict(kst=49),
], ids=str)
def test_select_refuses(lib, bad):
    assert _select(lib, **bad) == INVALID


def test_select_refuses_workspaces(lib):
    for w in (dict(ws=None), dict(ws=A + 16), dict(size=256)):
        assert _select(lib, **w) == WORKSPACE


def _compact(lib, pool=None, n=2, bt=A, mb=2, first=A, keep=A, ks=50, count=A, most=50, rotate=1,
             base=0.0, pair=0, ws=A, size=1 << 30):
    pool = pool or _pool()
    how = (base, pair) if isinstance(pool, kv.kv_quant_pool_desc) else (rotate,)
    return _f(lib, "kv_compact", pool)(C.byref(pool), n, bt, mb, first, keep, ks, count, most, *how,
                                       ws, size, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(bt=None), dict(bt=A + 2), dict(mb=-1), dict(mb=0), dict(first=A + 2),
    dict(keep=None), dict(keep=A + 1), dict(ks=49), dict(count=None), dict(most=-1),
    dict(rotate=2), dict(pool=_pool(rot_slot_stride=1028)), dict(pool=_mla_quant(), base=-1.0),
    dict(pool=_mla_quant(), base=NAN), dict(pool=_mla_quant(), pair=2),
    dict(n=1 << 30, most=1 << 20, ks=1 << 20),
], ids=str)
def test_compact_refuses(lib, bad):
    assert _compact(lib, **bad) == INVALID


def test_compact_refuses_shapes_and_workspaces(lib):
    assert _compact(lib, pool=_pool(rot_heads=2, copy_dim=256)) == UNSUPPORTED
    assert _compact(lib, pool=_quant(), base=1e4) == UNSUPPORTED  # e4m3 heads are not turned
    for w in (dict(ws=None), dict(ws=A + 16), dict(size=256)):
        assert _compact(lib, **w) == WORKSPACE


def test_binding_refuses_shapes():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    p = _pool()
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kv.kv_compact(p, i(2, 4), None, i(2, 5).float(), i(2), True, ws)
    with pytest.raises(ValueError):
        kv.kv_compact(p, i(3, 4), None, i(2, 5), i(2), True, ws)
    with pytest.raises(ValueError):
        kv.kv_compact(_mla_quant(), i(2, 4), None, i(2, 5), i(2), True, ws)
    with pytest.raises(ValueError):
        kv.kv_evict_select(torch.zeros(2, 9), i(2), i(3), 0, 0, i(2, 5), i(2), None, ws)
    with pytest.raises(ValueError):
        kv.kv_evict_select(torch.zeros(2, 9).double(), i(2), i(2), 0, 0, i(2, 5), i(2), None, ws)
    q, a = torch.zeros(8, 32, 128, dtype=torch.bfloat16), _attn()
    with pytest.raises(ValueError):
        kv.kv_attention_weights(p, 0, a, q, torch.zeros(8, 32), torch.zeros(2, 99), 1.0, ws)
    with pytest.raises(ValueError):
        kv.kv_attention_weights(p, 0, a, q.float(), torch.zeros(8, 32), torch.zeros(2, 100), 1.0, ws)
    with pytest.raises(ValueError):
        kv.kv_tree_attention(p, 0, a, i(7, 1), q, q.clone(), None, ws)
    with pytest.raises(ValueError):
        kv.kv_tree_attention(p, 0, a, i(8, 1).long(), q, q.clone(), None, ws)
    with pytest.raises(ValueError):
        kv.tree_mask([[0]])
