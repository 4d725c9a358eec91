"""Prefix sums of the 8-bit append and prompt attention that start below 0 or whose differences pass 32 bits: the
sequence is flagged and left out.  (2^31 - 1 to -2^31 would wrap to a count of one.)"""

import numpy as np
import pytest
import torch

from tests.fp8_util import Setup, bf16, f64

pytestmark = pytest.mark.gpu

KV_DEVERR_SEQ_RANGE = 3
HIGH, LOW = 2 ** 31 - 1, -2 ** 31


def cases(cu, most):
    for bad in ([-2, *cu[1:]], [HIGH, LOW, *cu[2:]], [LOW, HIGH, *cu[2:]], [HIGH, LOW, HIGH, cu[3]], [-5, -3, *cu[2:]]):
        yield bad, [b for b in range(3) if bad[b] >= 0 and 0 <= bad[b + 1] - bad[b] <= most]


def test_append(cuda_lib):
    count = [20, 33, 7]
    cu = np.concatenate([[0], np.cumsum(count)]).tolist()
    s = Setup(8, 2, 16, 3, 64, seed=1)
    q = bf16(s.rng.standard_normal((60, 8, 128)))
    k, v = (bf16(s.rng.standard_normal((60, 2, 128))) for _ in range(2))
    want_q = f64(s.append(q, k, v, [0] * 3, count))
    want = s.codes.cpu().numpy()
    for bad, kept in cases(cu, 33):
        s.codes.zero_()
        got = f64(s.append(q, k, v, [0] * 3, count, cu=bad, most=33))
        assert s.pool.error() == KV_DEVERR_SEQ_RANGE, bad
        for b in range(3):
            rows, pages = slice(cu[b], cu[b + 1]), s.table[b, :-(-count[b] // 16)]
            if b in kept:
                np.testing.assert_array_equal(got[rows], want_q[rows])
                np.testing.assert_array_equal(s.codes.cpu().numpy()[pages], want[pages])
            else:
                assert (got[rows] == 7).all() and not s.codes.cpu().numpy()[pages].any(), (bad, b)
    s.pool.close()


@pytest.mark.parametrize("count,n", [([20, 33, 7], [40, 33, 20]), ([3, 2, 4], [3000, 2000, 2500])])     # the second splits its keys
def test_prompts(cuda_lib, count, n):
    cu = np.concatenate([[0], np.cumsum(count)]).tolist()
    s = Setup(8, 2, 16, 3, max(n), seed=2)
    s.fill()
    q = bf16(s.rng.standard_normal((cu[-1], 8, 128)))
    want = s.prefill(q, count, n)
    for bad, kept in cases(cu, max(count)):
        out, lse = torch.full_like(q, 7.0), torch.full((cu[-1], 8), 7.0, device="cuda")
        out, lse = s.prefill(q, count, n, cu=np.array(bad), out=out, lse=lse)
        assert s.pool.error() == KV_DEVERR_SEQ_RANGE, bad
        for b in range(3):
            rows = slice(cu[b], cu[b + 1])
            if b in kept:
                np.testing.assert_array_equal(out[rows], want[0][rows])
                np.testing.assert_array_equal(lse[rows], want[1][rows])
            else:
                assert (out[rows] == 7).all() and (lse[rows] == 7).all(), (bad, b)
    s.pool.close()
