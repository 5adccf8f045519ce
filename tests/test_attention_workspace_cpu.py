"""Workspaces of kv_attention that serve several calls (no GPU: nothing is enqueued)."""
import pytest

import position_independent_mla_gb300 as kv
from position_independent_mla_gb300 import build as kbuild
from test_serve_abi_cpu import _attend, _attn, _pool, _quant

SLOTS = 64 * 100000
# (sequences, new tokens of each, cached tokens): a chunk that is split, one token, batches of
# many whole rows and of long contexts
CALLS = [(1, 16, 8192), (1, 1, 100), (1, 1, 10000), (64, 1, 16384), (8, 512, 8192), (200, 512, 8192)]


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kv.load()


def _call(n, q, k):
    return _attn(num_seqs=n, max_q_len=q, max_kv_len=k, max_blocks=k // 64 + 1)


@pytest.mark.parametrize("make", [_pool, _quant], ids=["bf16", "e4m3"])
def test_a_larger_calls_workspace_may_be_too_small_and_is_refused(lib, make):
    pool = make(num_slots=SLOTS)
    size = [kv.kv_attention_workspace_size(pool, _call(*c), c[0] * c[1], 32) for c in CALLS]
    assert size[0] > size[-1], "a split chunk needs more than a batch of 200 whole ones"
    for need, (n, q, k) in zip(size, CALLS):
        assert need >= 256 and need % 256 == 0
        for have in size:
            if have < need:
                assert _attend(lib, pool=pool, attn=_call(n, q, k), n=n * q,
                               size=have) == kv.KV_ERR_WORKSPACE
        assert _attend(lib, pool=pool, attn=_call(n, q, k), n=n * q,
                       size=need - 256) == kv.KV_ERR_WORKSPACE


@pytest.mark.parametrize("make", [_pool, _quant], ids=["bf16", "e4m3"])
def test_the_size_follows_from_the_stated_lengths_alone(lib, make):
    """Other pools, layers and device pointers: the same call, the same workspace."""
    for n, q, k in CALLS:
        a = kv.kv_attention_workspace_size(make(num_slots=SLOTS), _call(n, q, k), n * q, 32)
        b = kv.kv_attention_workspace_size(make(num_slots=2 * SLOTS, copy_layer_stride=4096 * 1024),
                                           _attn(num_seqs=n, max_q_len=q, max_kv_len=k,
                                                 max_blocks=k // 64 + 9, scale=2.0), n * q, 32)
        assert a == b
