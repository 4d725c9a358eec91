"""Decodes whose splits are joined through memory, for each group size: one long sequence of one and of three KV
heads, beside short ones of some, one and no tokens, against the fp64 models of the 8-bit and 4-bit caches."""

import numpy as np
import pytest

from tests import fp4_util, fp8_util
from tests.fp8_util import bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("util", [fp4_util, fp8_util])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("hkv,lens", [(1, [60001]), (1, [30000, 700]), (3, [20001]), (1, [16000, 1, 0, 300])])
def test_many_splits(cuda_lib, util, group, hkv, lens):
    hq = group * hkv
    s = util.Setup(hq, hkv, 16, len(lens), max(lens), seed=group)
    s.fill()
    q = bf16(s.rng.standard_normal((len(lens), hq, 128)))
    out, lse = s.decode(q, lens)
    s.check_rows(q, [(b, m - 1) for b, m in enumerate(lens)], out, lse, 0, 0, lens=lens)
    again = s.decode(q, lens)
    np.testing.assert_array_equal(again[0], out)
    np.testing.assert_array_equal(again[1], lse)
    assert s.pool.error() == 0
    s.pool.close()
