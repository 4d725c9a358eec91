"""What is left behind when a bounded wait of the 4-bit decode runs out: a warp's share of the tokens is skipped, and
nothing else."""

import math

import numpy as np
import pytest

from bit_kv_cache_12_gb300 import native
from tests.fp4_util import Setup, check_row
from tests.fp8_util import bf16, f64

pytestmark = pytest.mark.gpu

KV_DEVERR_TIMEOUT = 4
UNIT, WARPS = 32, 8                                            # tokens of a step; warps that take them in turns


def share(n, splits):
    """The tokens that the first warp of the first split has of a sequence of n."""
    units = -(-n // UNIT)
    per = -(-units // splits)
    lost = np.zeros(units * UNIT, bool)
    for u in range(0, per, WARPS):
        lost[u * UNIT:(u + 1) * UNIT] = True
    return lost[:n]


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("n", [5, 200, 3000, 20000])
def test_a_warp_that_gives_up(cuda_lib, hq, hkv, n):
    """Its share of the first sequence's first KV head is missing, whatever the number of splits; all else stands."""
    s = Setup(hq, hkv, 16, 2, n, seed=n)
    s.fill()
    q = bf16(s.rng.standard_normal((2, hq, 128)))
    lens = [n, 17 if n > 17 else 2]
    want, want_lse = s.decode(q, lens)
    native.kv_debug_stall_first_copy(s.pool.handle, 1, 200)
    out, lse = s.decode(q, lens)
    assert s.pool.error() == KV_DEVERR_TIMEOUT
    native.kv_debug_stall_first_copy(s.pool.handle, 0)
    G = hq // hkv
    np.testing.assert_array_equal(out[1], want[1])
    np.testing.assert_array_equal(lse[1], want_lse[1])
    np.testing.assert_array_equal(out[0, G:], want[0, G:])
    np.testing.assert_array_equal(lse[0, G:], want_lse[0, G:])
    k, v, ok = s.model.rows(s.table[0], n, 0)
    failed = {}
    for splits in range(1, 65):
        see = ok & ~share(n, splits)
        if see.tobytes() in failed:
            continue
        try:
            for h in range(G):
                check_row(out[0, h], lse[0, h], f64(q)[0, h], k, v, see, 1 / math.sqrt(128), (splits, h), 1.0)
            break
        except AssertionError as e:
            failed[see.tobytes()] = e
    else:
        raise AssertionError(list(failed.values()))
    again, again_lse = s.decode(q, lens)
    np.testing.assert_array_equal(again, want)
    np.testing.assert_array_equal(again_lse, want_lse)
    assert s.pool.error() == 0
    s.pool.close()


@pytest.mark.parametrize("polls", [1, 2, 3, 5])
def test_limits_that_run_out_as_copies_land(cuda_lib, polls):
    """Limits so short that copies land about when they run out: the call ends, says so if a wait ran out, is right if
    none did, and the next call with the usual limit is right."""
    s = Setup(16, 4, 16, 10, 3000, seed=polls)
    s.fill()
    q = bf16(s.rng.standard_normal((10, 16, 128)))
    n = s.rng.integers(1, 3001, 10).tolist()
    want, want_lse = s.decode(q, n, max_len=3000)
    for _ in range(20):
        native.kv_debug_stall_first_copy(s.pool.handle, 0, polls)
        out, lse = s.decode(q, n, max_len=3000)
        error = s.pool.error()
        assert error in (0, KV_DEVERR_TIMEOUT) and np.isfinite(out).all()
        if error == 0:
            np.testing.assert_array_equal(out, want)
            np.testing.assert_array_equal(lse, want_lse)
        native.kv_debug_stall_first_copy(s.pool.handle, 0, 0)
        out, lse = s.decode(q, n, max_len=3000)
        assert s.pool.error() == 0
        np.testing.assert_array_equal(out, want)
        np.testing.assert_array_equal(lse, want_lse)
    s.pool.close()
