"""Prompt attention kernels that give up with a full queue: a CTA has published four blocks of rows, holds a fifth
that it could not publish, and has asked the scheduler for another.  All of their rows are its own to account for."""

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from tests.fp8_util import Setup, bf16, f64, i32
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


def test_prefill_blocks_behind_a_full_queue(cuda_lib):
    """1,200 blocks with one pass each: the queue fills before the ring of passes does."""
    s = Setup(64, 8, 16, 150, 40, seed=22)
    s.fill(spread=0)
    count = [32] * 150
    n = s.rng.integers(32, 41, 150).tolist()
    q = bf16(s.rng.standard_normal((32 * 150, 64, 128)))
    cu, length, table = i32(np.arange(151) * 32), i32(n), i32(s.table)
    need = native.kv_prefill_workspace_bytes(s.pool.handle, 150, 32, 40)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(stalled):
        out = torch.full((q.shape[0], 64, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((q.shape[0], 64), 7.0, device="cuda")
        native.kv_debug_stall_first_copy(s.pool.handle, 2 if stalled else 0, 2000 if stalled else 0)
        native.kv_prefill_attention_fp8(s.pool.handle, 0, 150, q, cu, length, table, s.width, 32, 40, 0.1, 0, 0, out, lse, ws, need)
        torch.cuda.synchronize()
        assert s.pool.error() == (KV_DEVERR_TIMEOUT if stalled else 0)
        return f64(out), f64(lse)

    want, got, again = run(0), run(1), run(0)
    check(*got, *want, 8, 32)
    np.testing.assert_array_equal(again[0], want[0])
    np.testing.assert_array_equal(again[1], want[1])
    s.pool.close()
