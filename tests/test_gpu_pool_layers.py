"""More layers than the device holds: refused before the host's own storage of each layer is asked for."""

import ctypes
import resource

import pytest

from bit_kv_cache_12_gb300 import native as n

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [n.KV_POOL_INT2_3TIER, n.KV_POOL_BF16, n.KV_POOL_FP8, n.KV_POOL_FP4])
def test_layers_beyond_the_device(cuda_lib, kind):
    before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
    h = ctypes.c_void_p()
    cfg = n.KvPoolConfig(kind, 2 ** 31 - 1, 1, 1, 128, 16, 128, 64, 256, 1, 1)
    assert cuda_lib.kv_pool_create(ctypes.byref(cfg), None, ctypes.byref(h)) == n.KV_ERR_OOM
    assert not h.value
    assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 1 << 20     # KB
    pool = n.KVPool(kind, 1, 1, 1, 16, 1, 1)
    assert pool.error() == 0
    pool.close()
