"""What the 4-bit cache's entry points refuse on the host without a pool (no GPU)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_kv_cache_12_gb300 import build, native
    build.build()
    return native.lib()


def test_null_pools_are_refused(lib):
    from bit_kv_cache_12_gb300 import native as n
    f, bad = ctypes.c_float(1.0), n.KV_ERR_INVALID_ARG
    assert lib.kv_pool_get_fp4_layout(None, 0, None) == bad
    assert lib.kv_pool_set_fp4_range(None, 0, 0, 0) == bad
    assert lib.kv_pool_set_rope_axes(None, 0, 1, (ctypes.c_int32 * 1)(0), 1) == bad
    assert lib.kv_rope_apply_axes(None, 0, 1, None, 1, None, 0, None, 0, None, 0, None, 0, None) == bad
    assert lib.kv_append_fp4(None, 0, 1, None, 0, None, 0, None, None, None, 1, 1, None) == bad
    assert lib.kv_read_fp4(None, 0, 1, None, None, None, 1, 1, None, 0, None, 0, None) == bad
    assert lib.kv_decode_attention_fp4(None, 0, 1, None, None, None, 1, 1, f, 0, 0, None, None, None, 0, None) == bad
    assert lib.kv_prompt_attention(None, 1, None, 0, 0, None, 0, None, 0, 0, None, None, 1, 1, f, 0, 0, None, None, None, 0,
                                   None) == bad
    assert lib.kv_prompt_workspace_bytes(None, 1, 1, 1) == 0


def test_pool_configurations(lib):
    from bit_kv_cache_12_gb300 import native as n
    h = ctypes.c_void_p()

    def make(kind, hq, hkv, d, page):
        cfg = n.KvPoolConfig(kind, 1, hq, hkv, d, page, 128, 64, 256, 1, 10)
        return lib.kv_pool_create(ctypes.byref(cfg), None, ctypes.byref(h))
    assert make(5, 8, 2, 128, 16) == n.KV_ERR_INVALID_ARG
    assert make(n.KV_POOL_FP4, 8, 2, 64, 16) == n.KV_ERR_UNSUPPORTED
    assert make(n.KV_POOL_FP4, 8, 2, 128, 64) == n.KV_ERR_UNSUPPORTED
    assert make(n.KV_POOL_FP4, 6, 2, 128, 16) == n.KV_ERR_UNSUPPORTED
    assert make(n.KV_POOL_FP4, 7, 2, 128, 16) == n.KV_ERR_INVALID_ARG
