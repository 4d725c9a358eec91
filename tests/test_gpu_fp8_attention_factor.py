"""Factors on cos and sin: the ones that the cache's exponents can hold, and refusals of the others."""

import numpy as np
import pytest

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc
from tests.fp8_util import Setup, bf16, check_codes, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("factor", [1e39, 1e308, 1e19, 1024.0, 64.5, 1e-13, 1e-60, -1.0, float("inf"), float("nan")])
def test_refused(cuda_lib, factor):
    pool = native.KVPool(native.KV_POOL_FP8, 1, 1, 1, 16, 1, 1)
    with pytest.raises(native.KVError) as e:
        native.kv_pool_set_rope(pool.handle, 0, native.rope_config(attention_factor=factor))
    assert e.value.status == native.KV_ERR_INVALID_ARG
    pool.close()


def test_refused_where_the_scaling_gives_it(cuda_lib):
    pool = native.KVPool(native.KV_POOL_FP8, 1, 1, 1, 16, 1, 1)
    scaling = dict(scaling="yarn", original_max_position=4096)
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(factor=1e200, **scaling))
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(factor=1e300, attention_factor=1.0, **scaling))
    with pytest.raises(native.KVError):
        native.kv_pool_set_rope(pool.handle, 0, native.rope_config(factor=1e300, **scaling))
    pool.close()


@pytest.mark.parametrize("factor", [1e-12, 0.01, 1.0, 1.3, 64.0])
def test_exponents_and_codes(cuda_lib, factor):
    """Tiles of every size that bf16 holds, from zeros and subnormal squares to values that saturate."""
    s = Setup(hq=1, hkv=1, page=16, seqs=1, longest=16 * 60, rope=dict(rotary_dim=128, attention_factor=factor))
    size = np.exp2(np.linspace(-120, 120, 60)).repeat(16)[:, None, None]
    k = bf16(s.rng.standard_normal((960, 1, 128)) * size)
    v = bf16(s.rng.standard_normal((960, 1, 128)) * size)
    s.append(None, k, v, [0], [960])
    check_codes(s, fc.append(s.model, s.rope, f64(k), f64(v), [0], [960], s.table))
    s.pool.close()


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("factor", [1.0, 1.3, 64.0])
def test_the_largest_finite_rows_saturate(cuda_lib, style, factor):
    """Rows of +-3.3e38 at every angle: products with the factor would pass fp32's range, the stored values saturate."""
    s = Setup(hq=1, hkv=1, page=16, seqs=1, longest=200, rope=dict(rotary_dim=128, style=style, attention_factor=factor))
    k = bf16(3.3e38 * np.sign(s.rng.standard_normal((200, 1, 128))))
    s.append(None, k, k, [0], [200])
    check_codes(s, fc.append(s.model, s.rope, f64(k), f64(k), [0], [200], s.table))
    assert s.pool.error() == 0
    s.pool.close()
