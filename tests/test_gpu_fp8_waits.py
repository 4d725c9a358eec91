"""What is left behind when a bounded wait of the 8-bit attention kernels runs out."""

import numpy as np
import pytest

from bit_kv_cache_12_gb300 import native
from tests.fp8_util import Setup, bf16

pytestmark = pytest.mark.gpu

KV_DEVERR_TIMEOUT = 4


@pytest.mark.parametrize("polls", [1, 2, 3, 5])
def test_decode_limits_that_run_out_as_copies_land(cuda_lib, polls):
    """Limits so short that copies land about when they run out: the call ends, says so if a wait ran out, is
    right if none did, and the next call with the usual limit is right."""
    s = Setup(16, 4, 16, 40, 5000, seed=polls)
    s.fill()
    q = bf16(s.rng.standard_normal((40, 16, 128)))
    n = s.rng.integers(1, 5001, 40).tolist()
    want = s.decode(q, n, max_len=5000)
    for _ in range(20):
        native.kv_debug_stall_first_copy(s.pool.handle, 0, polls)
        out, lse = s.decode(q, n, max_len=5000)
        error = s.pool.error()
        assert error in (0, KV_DEVERR_TIMEOUT)
        assert np.isfinite(out).all()
        if error == 0:
            np.testing.assert_array_equal(out, want[0])
            np.testing.assert_array_equal(lse, want[1])
        native.kv_debug_stall_first_copy(s.pool.handle, 0, 0)
        out, lse = s.decode(q, n, max_len=5000)
        assert s.pool.error() == 0
        np.testing.assert_array_equal(out, want[0])
        np.testing.assert_array_equal(lse, want[1])
    s.pool.close()
