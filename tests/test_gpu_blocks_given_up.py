"""Prompt attention kernels that give up with a full queue: a CTA has published four blocks of rows, holds a fifth
that it could not publish, and has asked the scheduler for another.  All of their rows are its own to account for."""

import numpy as np
import pytest

from bit_kv_cache_12_gb300 import native
from tests.test_gpu_prompt import Prompt

pytestmark = pytest.mark.gpu

KV_DEVERR_TIMEOUT = 4
QUEUE = 4                                                      # blocks that a CTA publishes ahead


def check(out, lse, want, want_lse, hkv, tokens):
    """Rows (outputs of 7 before the call) are what they are in a call in order or not numbers; those of at least the
    queue's blocks and the fifth one are not, and of no more than those of one CTA."""
    lost = np.isnan(lse)
    np.testing.assert_array_equal(lost, np.isnan(out).all(-1))
    np.testing.assert_array_equal(lost, np.isnan(out).any(-1))
    np.testing.assert_array_equal(out[~lost], want[~lost])
    np.testing.assert_array_equal(lse[~lost], want_lse[~lost])
    heads = lost.reshape(len(lost), hkv, -1)
    assert (heads.all(-1) == heads.any(-1)).all()              # whole groups of heads
    assert QUEUE * tokens < heads.any(-1).sum() <= (QUEUE + 2) * tokens


def test_prompt_blocks_behind_a_full_queue(cuda_lib):
    """1,176 blocks of 32 queries, more than five to an SM; the first one's last values are never handed over."""
    p = Prompt(64, 8, [2400, 2300], [2400, 2900], seed=21)
    want, want_lse = p.run()
    native.kv_debug_stall_first_copy(p.pool.handle, True, 2000)
    out, lse = p.run()
    assert p.pool.error() == KV_DEVERR_TIMEOUT
    native.kv_debug_stall_first_copy(p.pool.handle, False)
    check(out, lse, want, want_lse, 8, 32)
    again, again_lse = p.run()
    np.testing.assert_array_equal(again, want)
    np.testing.assert_array_equal(again_lse, want_lse)
    p.close()
