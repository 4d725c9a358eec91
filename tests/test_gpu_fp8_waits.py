"""What is left behind when a bounded wait of the 8-bit attention kernels runs out."""

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from tests.fp8_util import Setup, bf16, f64, i32

pytestmark = pytest.mark.gpu

KV_DEVERR_TIMEOUT = 4


@pytest.mark.parametrize("polls", [1, 2, 3, 5])
def test_decode_limits_that_run_out_as_copies_land(cuda_lib, polls):
    """Limits so short that copies land about when they run out: the call ends, says so if a wait ran out, is
    right if none did, and the next call with the usual limit is right."""
    s = Setup(16, 4, 16, 10, 3000, seed=polls)
    s.fill()
    q = bf16(s.rng.standard_normal((10, 16, 128)))
    n = s.rng.integers(1, 3001, 10).tolist()
    want = s.decode(q, n, max_len=3000)
    for _ in range(20):
        native.kv_debug_stall_first_copy(s.pool.handle, 0, polls)
        out, lse = s.decode(q, n, max_len=3000)
        error = s.pool.error()
        assert error in (0, KV_DEVERR_TIMEOUT)
        assert np.isfinite(out).all()
        if error == 0:
            np.testing.assert_array_equal(out, want[0])
            np.testing.assert_array_equal(lse, want[1])
        native.kv_debug_stall_first_copy(s.pool.handle, 0, 0)
        out, lse = s.decode(q, n, max_len=3000)
        assert s.pool.error() == 0
        np.testing.assert_array_equal(out, want[0])
        np.testing.assert_array_equal(lse, want[1])
    s.pool.close()


def give_up(s, q, count, n, ws_value, window=0, sinks=0):
    """A prompt call whose first CTA gives up, into outputs of 7 and a workspace of `ws_value`; and the same call in order."""
    cu, length, table = i32(np.concatenate([[0], np.cumsum(count)])), i32(n), i32(s.table)
    most, longest = max(count), max(n)
    need = native.kv_prefill_workspace_bytes(s.pool.handle, len(count), most, longest)
    got = []
    for stalled in (1, 0):
        ws = torch.full((need // 4 + 4,), ws_value, device="cuda")
        out = torch.full((q.shape[0] + 5, s.hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((q.shape[0] + 5, s.hq), 7.0, device="cuda")
        native.kv_debug_stall_first_copy(s.pool.handle, stalled, 2000 if stalled else 0)
        native.kv_prefill_attention_fp8(s.pool.handle, 0, len(count), q, cu, length, table, s.width, most, longest, 0.1,
                                        window, sinks, out, lse, ws, need)
        torch.cuda.synchronize()
        assert s.pool.error() == (KV_DEVERR_TIMEOUT if stalled else 0)
        got += [f64(out), f64(lse)]
    out, lse, want, want_lse = got
    lost = np.isnan(lse)
    np.testing.assert_array_equal(lost, np.isnan(out).all(-1))
    np.testing.assert_array_equal(lost, np.isnan(out).any(-1))
    np.testing.assert_array_equal(out[~lost], want[~lost])
    np.testing.assert_array_equal(lse[~lost], want_lse[~lost])
    return lost


def test_prefill_block_that_gives_up(cuda_lib):
    """Its rows, which it had begun, are not numbers; all others stand, and nobody's rows are left alone."""
    s = Setup(8, 2, 16, 2, 600, seed=2)
    s.fill()
    q = bf16(s.rng.standard_normal((400, 8, 128)))
    lost = give_up(s, q, [300, 100], [600, 100], 3.0)
    mine = np.zeros_like(lost)
    mine[256:300, :4] = True                                   # the first item: the last block of the first sequence, KV head 0
    np.testing.assert_array_equal(lost, mine)
    s.pool.close()


@pytest.mark.parametrize("window,sinks", [(0, 0), (4096, 64)])
def test_prefill_split_that_gives_up(cuda_lib, window, sinks):
    """Keys split over CTAs: the rows that miss a part are not numbers, whatever the workspace held."""
    s = Setup(8, 2, 16, 1, 9000, seed=3)
    s.fill()
    q = bf16(s.rng.standard_normal((3, 8, 128)))
    for value in (0.0, 3.0, -3e38):
        lost = give_up(s, q, [3], [9000], value, window, sinks)
        mine = np.zeros_like(lost)
        mine[:3, :4] = True
        np.testing.assert_array_equal(lost, mine)
    s.pool.close()


def test_prefill_blocks_taken_on_and_given_up(cuda_lib):
    """More blocks than SMs: the CTA that gives up has asked for another block ahead; its rows are not numbers either."""
    s = Setup(16, 2, 16, 2, 3400, seed=4)
    s.fill()
    q = bf16(s.rng.standard_normal((5200, 16, 128)))
    lost = give_up(s, q, [3000, 2200], [3400, 2200], 3.0)
    assert lost[2976:3000, :8].all()                           # the first item, 24 queries
    heads = lost.reshape(-1, 2, 8)
    assert (heads.all(-1) == heads.any(-1)).all()              # whole groups of heads,
    assert 0 < heads.any(-1).sum() <= 24 + 32                  # of two blocks of 32 queries at most
    s.pool.close()


def test_prefill_bound_on_queries_far_above_their_number(cuda_lib):
    """Blocks without rows take longer to pass over than a wait may last (here by a short limit; with the usual one from
    about 10^9 blocks on, which the calls allow): no wait runs out, and every row is written."""
    s = Setup(8, 8, 16, 16, 300, seed=5)
    s.fill()
    count = s.rng.integers(1, 40, 16).tolist()
    n = [int(s.rng.integers(c, 301)) for c in count]
    q = bf16(s.rng.standard_normal((sum(count), 8, 128)))
    want = s.prefill(q, count, n)
    native.kv_debug_stall_first_copy(s.pool.handle, 0, 300)    # about a millisecond
    for _ in range(2):
        out, lse = s.prefill(q, count, n, most=6553600)        # 3.3 million blocks: about ten
        assert s.pool.error() == 0
        np.testing.assert_array_equal(out, want[0])
        np.testing.assert_array_equal(lse, want[1])
    s.pool.close()


def test_limits_too_short_to_outlast_copies_are_refused(cuda_lib):
    """The INT2 and BF16 decodes wait for copies in flight with the hook's limit."""
    for kind in (native.KV_POOL_INT2_3TIER, native.KV_POOL_BF16):
        pool = native.KVPool(kind, 1, 4, 2, 16, 4, 1)
        for polls in (1, 100, 1023):
            for enable in (0, 1):
                with pytest.raises(native.KVError) as e:
                    native.kv_debug_stall_first_copy(pool.handle, enable, polls)
                assert e.value.status == native.KV_ERR_INVALID_ARG
        native.kv_debug_stall_first_copy(pool.handle, 1, 1024)
        native.kv_debug_stall_first_copy(pool.handle, 0, 0)
        pool.close()
