"""The bounded waits of the 8-bit attention kernels: a wait that runs out sets the
error word, ends the launch and leaves the pool usable."""

import numpy as np
import pytest

from bit_kv_cache_12_gb300 import native
from tests.fp8_util import Setup, bf16

pytestmark = pytest.mark.gpu

KV_DEVERR_TIMEOUT = 4


def test_decode_wait_runs_out(cuda_lib):
    s = Setup(8, 2, 16, 2, 3000, seed=1)
    s.fill()
    q = bf16(s.rng.standard_normal((2, 8, 128)))
    want = s.decode(q, [3000, 700])
    native.kv_debug_stall_first_copy(s.pool.handle, 1, 2000)
    out, lse = s.decode(q, [3000, 700])
    assert s.pool.error() == KV_DEVERR_TIMEOUT
    np.testing.assert_array_equal(out[0, 4:], want[0][0, 4:])          # the other KV heads and sequences stand
    np.testing.assert_array_equal(out[1], want[0][1])
    native.kv_debug_stall_first_copy(s.pool.handle, 0, 0)
    again = s.decode(q, [3000, 700])
    np.testing.assert_array_equal(again[0], want[0])
    np.testing.assert_array_equal(again[1], want[1])
    assert s.pool.error() == 0
    s.pool.close()


def test_prefill_wait_runs_out(cuda_lib):
    s = Setup(8, 2, 16, 2, 600, seed=2)
    s.fill()
    count, n = [300, 100], [600, 100]
    q = bf16(s.rng.standard_normal((400, 8, 128)))
    want = s.prefill(q, count, n)
    native.kv_debug_stall_first_copy(s.pool.handle, 1, 2000)
    out, lse = s.prefill(q, count, n)
    assert s.pool.error() == KV_DEVERR_TIMEOUT
    lost = np.isnan(out).any(-1)
    assert lost.any() and not lost[:, 4:].any()                        # rows of one block of one KV head
    np.testing.assert_array_equal(out[~lost], want[0][~lost])
    native.kv_debug_stall_first_copy(s.pool.handle, 0, 0)
    again = s.prefill(q, count, n)
    np.testing.assert_array_equal(again[0], want[0])
    np.testing.assert_array_equal(again[1], want[1])
    assert s.pool.error() == 0
    s.pool.close()
