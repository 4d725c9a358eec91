"""Pools beyond any device's memory, whose sizes in bytes pass 64 bits, are refused before anything is allocated."""

import ctypes

import pytest

from bit_kv_cache_12_gb300 import build, native as n


@pytest.mark.parametrize("kind", [n.KV_POOL_INT2_3TIER, n.KV_POOL_BF16, n.KV_POOL_FP8, n.KV_POOL_FP4])
@pytest.mark.parametrize("layers,heads,pages,seqs", [(1, 1 << 29, 1 << 27, 1), (1 << 20, 1 << 20, 1 << 24, 1),
                                                     (1, 1 << 30, 1 << 30, 1 << 30), (1 << 20, 1 << 20, 1, 1 << 20)])
def test_sizes_beyond_64_bits(kind, layers, heads, pages, seqs):
    build.build()
    h = ctypes.c_void_p()
    cfg = n.KvPoolConfig(kind, layers, heads, heads, 128, 16, 128, 64, 256, seqs, pages)
    assert n.lib().kv_pool_create(ctypes.byref(cfg), None, ctypes.byref(h)) == n.KV_ERR_OOM
    assert not h.value
