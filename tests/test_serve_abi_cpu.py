"""Argument checks of the quantised-row and attention calls (no GPU: every
call here is refused before anything is enqueued)."""
import ctypes as C

import pytest
import torch

import position_independent_mla_gb300 as kv
from position_independent_mla_gb300 import build as kbuild

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kv.load()


def _pool(**k):
    d = dict(num_layers=2, block_size=64, num_slots=128, copy_base=A, copy_layer_stride=128 * 1024,
             copy_slot_stride=1024, copy_dim=1024, rot_base=A, rot_layer_stride=128 * 1024,
             rot_slot_stride=1024, rot_heads=8, rot_head_dim=128, rope_base=1e4, pair_convention=0)
    d.update(k)
    return kv.kv_pool_desc(**d)


def _quant(**k):
    d = dict(num_layers=2, block_size=64, num_slots=128, copy_base=A, copy_layer_stride=128 * 1024,
             copy_slot_stride=1024, copy_dim=1024, copy_scale=A, copy_scale_layer_stride=1024,
             copy_scale_slot_stride=8, rot_base=A, rot_layer_stride=128 * 1024,
             rot_slot_stride=1024, rot_heads=8, rot_head_dim=128, rot_scale=A,
             rot_scale_layer_stride=1024, rot_scale_slot_stride=8)
    d.update(k)
    return kv.kv_quant_pool_desc(**d)


def _attn(**k):
    d = dict(num_seqs=2, max_q_len=4, max_kv_len=100, max_blocks=2, d_q_off=A, d_kv_len=A,
             d_block_tables=A, causal=1, window=0, sinks=0, scale=0.1)
    d.update(k)
    return kv.kv_attn_desc(**d)


def _attend(lib, pool=None, layer=0, attn=None, n=8, heads=32, q=A, qs=(4096, 128), out=A,
            os=(4096, 128), lse=A, ws=A, size=1 << 30):
    pool = pool or _pool()
    f = lib.kv_attention_quant if isinstance(pool, kv.kv_quant_pool_desc) else lib.kv_attention
    return f(C.byref(pool), layer, C.byref(attn or _attn()), n, heads, q, *qs, out, *os, lse, ws,
             size, None)


@pytest.mark.parametrize("bad", [
    dict(layer=2), dict(layer=-1), dict(heads=0), dict(heads=33), dict(n=-1), dict(n=9),
    dict(q=None), dict(q=A + 8), dict(out=None), dict(out=A + 2), dict(qs=(4096, 4)),
    dict(qs=(-8, 128)), dict(os=(4095, 128)), dict(lse=A + 2),
    dict(pool=_pool(num_slots=100)), dict(pool=_pool(copy_base=None)),
    dict(pool=_pool(rot_slot_stride=1028)), dict(pool=_quant(copy_slot_stride=1032)),
    dict(pool=_quant(copy_scale=None)), dict(pool=_quant(rot_base=A + 8)),
    dict(attn=_attn(num_seqs=-1)), dict(attn=_attn(causal=2)), dict(attn=_attn(window=-1)),
    dict(attn=_attn(sinks=-1)), dict(attn=_attn(window=5, causal=0)), dict(attn=_attn(scale=0.0)),
    dict(attn=_attn(scale=-1.0)), dict(attn=_attn(scale=float("nan"))),
    dict(attn=_attn(scale=float("inf"))), dict(attn=_attn(d_q_off=None)),
    dict(attn=_attn(d_kv_len=A + 1)), dict(attn=_attn(d_block_tables=None)),
    dict(attn=_attn(max_blocks=0)),
], ids=str)
def test_attention_refuses(lib, bad):
    assert _attend(lib, **bad) == kv.KV_ERR_INVALID_ARG


def test_attention_refuses_other_shapes_and_small_workspaces(lib):
    assert _attend(lib, pool=_pool(copy_dim=256, rot_heads=2)) == kv.KV_ERR_UNSUPPORTED
    mla = dict(copy_dim=512, rot_heads=1, rot_head_dim=64)
    assert _attend(lib, pool=_pool(**mla), heads=129) == kv.KV_ERR_UNSUPPORTED
    # k_pe in e4m3, or head keys in bf16 beside e4m3 values, has no kernel
    assert _attend(lib, pool=_quant(**mla)) == kv.KV_ERR_UNSUPPORTED
    assert _attend(lib, pool=_quant(rot_scale=None)) == kv.KV_ERR_UNSUPPORTED
    for ws, size in ((None, 1 << 30), (A + 16, 1 << 30), (A, 16)):
        assert _attend(lib, ws=ws, size=size) == kv.KV_ERR_WORKSPACE
    assert lib.kv_attention(None, 0, None, 1, 1, A, 8, 8, A, 8, 8, A, A, 1 << 30,
                            None) == kv.KV_ERR_INVALID_ARG
    assert lib.kv_attention(C.byref(_pool()), 0, None, 1, 32, A, 8, 8, A, 8, 8, A, A, 1 << 30,
                            None) == kv.KV_ERR_INVALID_ARG


def test_attention_workspace_sizes(lib):
    n = kv.kv_attention_workspace_size(_pool(), _attn(), 8, 32)
    assert n >= 256 and n % 256 == 0
    assert kv.kv_attention_workspace_size(_quant(), _attn(), 8, 32) >= 256
    assert kv.kv_attention_workspace_size(_pool(), _attn(scale=0.0), 8, 32) == 0
    assert kv.kv_attention_workspace_size(_pool(num_slots=1), _attn(), 8, 32) == 0


def _quantize(lib, src=None, slots=None, dst=None, layer=0, n=10, at=A, ws=A, size=1 << 20):
    return lib.kv_quantize(C.byref(src or _pool()), slots, C.byref(dst or _quant()), layer, n, at,
                           ws, size, None)


@pytest.mark.parametrize("bad", [
    dict(layer=1), dict(layer=-1), dict(n=-1), dict(n=129), dict(at=None), dict(at=A + 2),
    dict(slots=A + 1), dict(src=_pool(copy_dim=512, rot_heads=4)), dict(src=_pool(rot_base=None)),
    dict(dst=_quant(copy_dim=1000)), dict(dst=_quant(copy_scale=A + 2)),
    dict(dst=_quant(num_layers=0)), dict(dst=_quant(copy_scale_slot_stride=-1)),
], ids=str)
def test_quantize_refuses(lib, bad):
    assert _quantize(lib, **bad) == kv.KV_ERR_INVALID_ARG
    k = dict(bad)
    src, slots, dst = k.pop("src", None), k.pop("slots", None), k.pop("dst", None)
    assert lib.kv_dequantize(C.byref(dst or _quant()), k.get("layer", 0), k.get("at", A),
                             C.byref(src or _pool()), k.get("n", 10), slots, A, 1 << 20,
                             None) == kv.KV_ERR_INVALID_ARG


def test_quantize_refuses_other_shapes_and_small_workspaces(lib):
    assert _quantize(lib, dst=_quant(rot_scale=None)) == kv.KV_ERR_UNSUPPORTED
    assert _quantize(lib, ws=None) == kv.KV_ERR_WORKSPACE
    assert _quantize(lib, size=255) == kv.KV_ERR_WORKSPACE
    assert kv.load().kv_quantize_workspace_size(C.byref(_quant(copy_dim=0))) == 0


def test_python_checks_of_tensor_shapes():
    q = torch.zeros(8, 32, 128, dtype=torch.bfloat16)
    lse = torch.zeros(8, 32)
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    for bad in (dict(q=q.float()), dict(q=q[..., :64]), dict(q=q.transpose(1, 2)),
                dict(out=q[:4]), dict(out=q.half()), dict(lse=lse.double()), dict(lse=lse.t())):
        args = dict(q=q, out=q, lse=lse)
        args.update(bad)
        with pytest.raises(ValueError):
            kv.kv_attention(_pool(), 0, _attn(), args["q"], args["out"], args["lse"], ws)
    with pytest.raises(kv.KVError):
        kv.kv_attention(_pool(), 5, _attn(), q, q, lse, ws)
