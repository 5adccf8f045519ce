"""Quantised rows on the GPU: written values and scales against the 64-bit
form bit for bit, and read back exactly."""
import math

import pytest
import torch

import position_independent_mla_gb300 as kv
from _serve import SHAPES, bf16_rows, empty_quant, ref_quantize, value64

pytestmark = pytest.mark.gpu


def _src(kind, layers, rows, seed, special=False):
    cd, h, d, base = SHAPES[kind]
    g = torch.Generator().manual_seed(seed)
    copy, rot = bf16_rows(g, layers, rows, cd), bf16_rows(g, layers, rows, h * d)
    if special:
        copy[0, 0, :128] = 0.0                       # an empty group
        copy[0, 0, 128] = math.nan
        copy[0, 0, 129] = math.inf
        copy[0, 0, 130] = -math.inf
        copy[0, 1, 256:384] = 2.0 ** -130            # subnormal: the smallest scale
        copy[0, 1, 384] = 3.0e38                     # the largest scale
        copy[0, 2, :128] *= 2.0 ** -60
        copy[0, 2, 128:256] *= 2.0 ** 80
        copy[0, 3, 0] = 448.0 * 4                    # exactly at a power's limit
        copy[0, 3, 1:128] = 0.25
        copy[0, 3, 128] = 449.0 * 4                  # rounds to 1792 in bf16: the same limit
        copy[0, 3, 256] = 456.0 * 4                  # above it
        copy[0, 3, 384:512] = math.nan               # nothing finite
    return copy, rot, base


@pytest.mark.parametrize("kind", sorted(SHAPES))
@pytest.mark.parametrize("layers,rows,pad", [(1, 1, 0), (1, 33, 1), (3, 130, 0)])
def test_quantize_and_back(kind, layers, rows, pad):
    cd, h, d, _ = SHAPES[kind]
    copy, rot, base = _src(kind, layers, rows, rows, special=rows > 4)
    slots = 64 * (rows // 64 + 2)
    p = empty_quant(kind, layers + 2, slots, 64, pad)
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(5))[:rows].int().cuda()
    src = kv.pool_desc(copy.cuda(), rot.cuda(), 1, h, base)
    ws = kv.quant_workspace(p.desc)
    kv.kv_quantize(src, None, p.desc, 1, rows, at, ws)
    assert kv.kv_get_device_status(ws) == kv.KV_OK and kv.kv_last_launch_count() == 1
    want_c, want_s = ref_quantize(copy)
    got = p.copy[1:1 + layers, at.long()].float().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want_c))
    assert torch.equal(got.nan_to_num(), want_c.nan_to_num())
    assert torch.equal(p.copy_scale[1:1 + layers, at.long()].cpu().double(), want_s)
    if kind == "mla":
        assert torch.equal(p.rot[1:1 + layers, at.long()].cpu(), rot)
    else:
        want, sc = ref_quantize(rot)
        assert torch.equal(p.rot[1:1 + layers, at.long()].float().cpu().double(), want)
        assert torch.equal(p.rot_scale[1:1 + layers, at.long()].cpu().double(), sc)
    # layers and slots that were not named stay as they were
    rest = torch.ones(slots, dtype=torch.bool)
    rest[at.long().cpu()] = False
    assert not p.copy[0].float().any() and not p.copy[-1].float().any()
    assert not p.copy[1:-1, rest.cuda()].float().any()

    back_c = torch.zeros(layers, slots, cd, dtype=torch.bfloat16, device="cuda")
    back_r = torch.zeros(layers, slots, h * d, dtype=torch.bfloat16, device="cuda")
    dst = kv.pool_desc(back_c, back_r, 64, h, base)
    to = torch.randperm(slots, generator=torch.Generator().manual_seed(6))[:rows].int().cuda()
    kv.kv_dequantize(p.desc, 1, at, dst, rows, to, ws)
    assert kv.kv_get_device_status(ws) == kv.KV_OK
    v = value64(p.copy[1:1 + layers, at.long()], p.copy_scale[1:1 + layers, at.long()])
    g = back_c[:, to.long()].double()
    assert torch.equal(torch.isnan(g), torch.isnan(v)) and torch.equal(g.nan_to_num(), v.nan_to_num())
    r = value64(p.rot[1:1 + layers, at.long()],
                None if kind == "mla" else p.rot_scale[1:1 + layers, at.long()])
    assert torch.equal(back_r[:, to.long()].double(), r)


def test_source_slots_other_stream_and_reused_workspace():
    copy, rot, base = _src("mla", 2, 64, 9)
    p = empty_quant("mla", 2, 64, 64)
    src = kv.pool_desc(copy.cuda(), rot.cuda(), 64, 1, base)
    a = torch.randperm(64, generator=torch.Generator().manual_seed(1))[:17].int().cuda()
    b = torch.randperm(64, generator=torch.Generator().manual_seed(2))[:17].int().cuda()
    ws = torch.full_like(kv.quant_workspace(p.desc), 255)  # whatever it held before
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kv.kv_quantize(src, a, p.desc, 0, 17, b, ws, stream=st)
    assert kv.kv_get_device_status(ws, st) == kv.KV_OK
    want, _ = ref_quantize(copy[:, a.long().cpu()])
    assert torch.equal(p.copy[:, b.long()].float().cpu().double(), want)


def test_bad_slots_are_reported_and_skipped():
    copy, rot, base = _src("gqa4", 1, 8, 3)
    p = empty_quant("gqa4", 1, 64, 64)
    src = kv.pool_desc(copy.cuda(), rot.cuda(), 1, 4, base)
    at = torch.tensor([3, -1, 5, 64, 7, 8, 9, 10], dtype=torch.int32, device="cuda")
    ws = kv.quant_workspace(p.desc)
    kv.kv_quantize(src, None, p.desc, 0, 8, at, ws)
    assert kv.kv_get_device_status(ws) == kv.KV_ERR_OUT_OF_RANGE
    want, _ = ref_quantize(copy)
    ok = [0, 2, 4, 5, 6, 7]
    assert torch.equal(p.copy[0, at[ok].long()].float().cpu().double(), want[0, ok])
    kv.kv_quantize(src, None, p.desc, 0, 1, at, ws)  # the next call reports for itself
    assert kv.kv_get_device_status(ws) == kv.KV_OK
    kv.kv_quantize(src, None, p.desc, 0, 0, at, ws)
    assert kv.kv_get_device_status(ws) == kv.KV_OK
