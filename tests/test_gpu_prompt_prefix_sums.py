"""Prefix sums of prompts whose differences pass 32 bits: the sequence is flagged and left out, as any other that is
not in order.  (2^31 - 1 to -2^31 would wrap to a count of one.)"""

import numpy as np
import pytest

from tests.test_gpu_prompt import Prompt

pytestmark = pytest.mark.gpu

KV_DEVERR_SEQ_RANGE = 3
HIGH, LOW = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("count,keys", [([20, 33, 7], [40, 33, 20]), ([3, 2, 4], [3000, 2000, 2500])])   # the second splits its keys
def test_differences_beyond_32_bits(cuda_lib, count, keys):
    p = Prompt(8, 2, count, keys, seed=9)
    want = p.run()
    p.check(*want, sample=20)
    cq, ck = p.cq.tolist(), p.ck.tolist()
    for which, bad in (("cq", [HIGH, LOW, *cq[2:]]), ("cq", [LOW, HIGH, *cq[2:]]), ("ck", [HIGH, LOW, *ck[2:]]),
                       ("ck", [LOW, HIGH, *ck[2:]]), ("cq", [HIGH, LOW, HIGH, cq[3]]), ("ck", [LOW, LOW, ck[2], ck[3]])):
        out, lse = p.run(**{which: bad})
        assert p.pool.error() == KV_DEVERR_SEQ_RANGE, bad
        sums = np.array(bad)
        kept = [b for b in range(3) if sums[b] >= 0 and 0 <= sums[b + 1] - sums[b] <= (max(count) if which == "cq" else max(keys))]
        for b in range(3):
            part = slice(int(p.cq[b]), int(p.cq[b + 1]))
            if b in kept:
                np.testing.assert_array_equal(out[part], want[0][part])
                np.testing.assert_array_equal(lse[part], want[1][part])
            else:
                assert (out[part] == 7).all() and (lse[part] == 7).all(), (bad, b)
    p.close()
