"""What the 8-bit cache's entry points refuse on the host, without a GPU: a pool
handle cannot be made here, so these are the checks that come before one is
used, and the rotary configuration's arithmetic."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_kv_cache_12_gb300 import build, native
    build.build()
    return native.lib()


def test_null_pools_are_refused(lib):
    from bit_kv_cache_12_gb300 import native as n
    f = ctypes.c_float(1.0)
    bad = n.KV_ERR_INVALID_ARG
    assert lib.kv_pool_get_fp8_layout(None, 0, None) == bad
    assert lib.kv_pool_set_rope(None, 0, ctypes.byref(n.rope_config())) == bad
    assert lib.kv_rope_apply(None, 0, 1, None, None, 0, None, 0, None, 0, None, 0, None) == bad
    assert lib.kv_append_fp8(None, 0, 1, None, 0, None, 0, None, 0, None, None, None, 1, 1, None, None) == bad
    assert lib.kv_decode_attention_fp8(None, 0, 1, None, None, None, 1, 1, f, 0, 0, None, None, None, 0, None) == bad
    assert lib.kv_prefill_attention_fp8(None, 0, 1, None, None, None, None, 1, 1, 1, f, 0, 0, None, None, None, 0,
                                        None) == bad
    assert lib.kv_prefill_workspace_bytes(None, 1, 1, 1) == 0


def test_pool_configurations(lib):
    from bit_kv_cache_12_gb300 import native as n
    h = ctypes.c_void_p()

    def make(kind, hq, hkv, d, page):
        cfg = n.KvPoolConfig(kind, 1, hq, hkv, d, page, 128, 64, 256, 1, 10)
        return lib.kv_pool_create(ctypes.byref(cfg), None, ctypes.byref(h))
    assert make(3, 8, 2, 128, 16) == n.KV_ERR_INVALID_ARG
    assert make(n.KV_POOL_FP8, 8, 2, 64, 16) == n.KV_ERR_UNSUPPORTED
    assert make(n.KV_POOL_FP8, 8, 2, 128, 64) == n.KV_ERR_UNSUPPORTED
    assert make(n.KV_POOL_FP8, 6, 2, 128, 16) == n.KV_ERR_UNSUPPORTED
    assert make(n.KV_POOL_FP8, 7, 2, 128, 16) == n.KV_ERR_INVALID_ARG


def test_rope_config_checks_the_speeds_count():
    from bit_kv_cache_12_gb300 import native as n
    with pytest.raises(ValueError):
        n.rope_config(rotary_dim=64, inv_freq=[1.0] * 31)
    with pytest.raises(KeyError):
        n.rope_config(style="other")
