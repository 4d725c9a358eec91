"""Windows and counts of first tokens up to the largest integer, and prompts without a key, over the 4-bit cache and
over packed rows."""

import math

import numpy as np
import pytest

from tests.fp4_util import Setup
from tests.fp8_util import bf16
from tests.test_gpu_prompt import Prompt

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1
WINDOWS = [1, 16, 299, 300, 301, TOP - 1, TOP]
SINKS = [0, 1, 31, 300, TOP]


@pytest.mark.parametrize("window", WINDOWS)
def test_decode(cuda_lib, window):
    s = Setup(8, 2, 16, 3, 300, seed=window % 97)
    s.fill()
    q = bf16(s.rng.standard_normal((3, 8, 128)))
    n = [300, 17, 299]
    for sinks in SINKS:
        out, lse = s.decode(q, n, window, sinks)
        s.check_rows(q, [(b, m - 1) for b, m in enumerate(n)], out, lse, window, sinks, lens=n)
    assert s.pool.error() == 0
    s.pool.close()


@pytest.mark.parametrize("window", WINDOWS)
def test_prompt(cuda_lib, window):
    p = Prompt(8, 2, [300, 5, 40], [300, 300, 33], seed=window % 89)        # the last: more queries than keys
    for sinks in SINKS:
        p.check(*p.run(window, sinks), window, sinks, sample=60)
    p.close()


def test_prompt_without_keys(cuda_lib):
    p = Prompt(8, 2, [300, 5], [0, 0], seed=1)
    for window, sinks in ((0, 0), (7, 3), (TOP, TOP)):
        out, lse = p.run(window, sinks)
        assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = p.run(kv_rows=1)
    assert not np.any(out) and np.isneginf(lse).all()
    p.close()
