"""The 8-bit attention where a logit's own rounding in fp32 is as large as the range of the fp16
weights: the output stays a mean of the visible values, and the value of the largest logit where
no other is near."""

import math

import numpy as np
import pytest

from oracle import fp8cache as fc
from tests.fp8_util import Setup, bf16, f64

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)


def check(s, q, rows, out, lse, window, scale):
    """Against the fp64 model, and for each row: inside the span of the visible values, and where one
    logit leads by more than every error, that key's value alone.

    Span: bf16 of a mean whose weights are rounded to fp16: 2^-8 + 2^-11 and the sums' fp32.  Alone:
    the other weights are below 2^-25 of it; value (4 bits) * fp16 weight / fp32 weight is off by
    2^-11 and rounds back to the value in bf16."""
    s.check_rows(q, rows, out, lse, window, 0, scale, lens=[s.length] * s.seqs)
    q = f64(q)
    G, alone = s.hq // s.hkv, 0
    for i, (b, pos) in enumerate(rows):
        for h in range(s.hq):
            k, v, ok = s.model.rows(s.table[b], s.length, h // G)
            see = fc.visible(pos, s.length, window, 0)
            k, v = k[see], v[see]
            x = k @ q[i, h] * scale
            top = np.argsort(x)[::-1]
            error = 2.0 ** -18 * float(np.max(np.abs(k) @ np.abs(q[i, h])) * abs(scale)) + 2.0 ** -22
            slack = (2.0 ** -8 + 2.0 ** -10) * np.abs(v).max(0)
            assert np.all(out[i, h] >= v.min(0) - slack) and np.all(out[i, h] <= v.max(0) + slack), (i, h, pos)
            if len(x) == 1 or x[top[0]] - x[top[1]] > 2 * error + 25:
                np.testing.assert_array_equal(out[i, h], v[top[0]], err_msg=str((i, h, pos)))
                alone += 1
    return alone


def powers(rng, shape):
    """Query sizes 2^0 to 2^105, most of them where logits pass 2^20."""
    return np.exp2(rng.integers(0, 106, shape).astype(float))


@pytest.mark.parametrize("window", [1, 2, 17, 0])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (8, 8)])
def test_decode(cuda_lib, window, hq, hkv):
    s = Setup(hq, hkv, 16, 40, 70, seed=window)
    s.length = 70
    s.fill(spread=3)
    if window < 2:                                        # one key: every exponent of V
        s.model.exps[..., 1] = s.rng.integers(-64, 8, s.model.exps.shape[:-1])
        s.upload()
    for scale in (SCALE, -3.0):
        q = bf16(s.rng.standard_normal((40, hq, 128)) * powers(s.rng, (40, hq, 1)))
        out, lse = s.decode(q, [70] * 40, window, 0, scale)
        assert check(s, q, [(b, 69) for b in range(40)], out, lse, window, scale) > 40
    s.pool.close()


@pytest.mark.parametrize("window", [1, 2, 17, 0])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2)])
def test_prefill(cuda_lib, window, hq, hkv):
    s = Setup(hq, hkv, 16, 1, 200, seed=window)
    s.length = 200
    s.fill(spread=3)
    for scale in (SCALE, -3.0):
        size = powers(s.rng, (90, hq, 1))
        size[:20], size[20:40, 0] = 1.0, 2.0 ** 40        # a warp of ordinary rows, and some of both kinds
        q = s.rng.standard_normal((90, hq, 128))
        out, lse = s.prefill(bf16(q * size), [90], [200], window, 0, scale)
        assert check(s, bf16(q * size), [(0, 110 + i) for i in range(90)], out, lse, window, scale) > 40
        # a row does not depend on the rows beside it
        small = size == 1.0
        again = s.prefill(bf16(q * np.where(small, 1.0, 1.5)), [90], [200], window, 0, scale)
        pick = np.broadcast_to(small, (90, hq, 1))[..., 0]
        np.testing.assert_array_equal(out[pick], again[0][pick])
        np.testing.assert_array_equal(lse[pick], again[1][pick])
    s.pool.close()


@pytest.mark.parametrize("power", [22, 25, 28, 31, 60])
def test_all_logits_large_and_negative(cuda_lib, power):
    """Every logit near -2^power, rising along the cache: the reference follows downwards too."""
    s = Setup(4, 1, 16, 1, 300, seed=power)
    s.length = 300
    s.fill(spread=0)
    s.model.exps[..., 0] = 0
    k_at, _ = fc.places()
    for j in range(300):
        code = fc.e4m3_encode(fc.e4m3_round(np.full(128, 448.0 - j)))
        s.model.codes[s.table[0][j // 16], 0, 0, 0][k_at[j % 16]] = code
    s.upload()
    q = bf16(np.full((60, 4, 128), -2.0 ** (power - 13)))
    one = q[59:].contiguous()
    out, lse = s.decode(one, [300], 0, 0, SCALE)
    check(s, one, [(0, 299)], out, lse, 0, SCALE)
    out, lse = s.prefill(q, [60], [300], 0, 0, SCALE)
    check(s, q, [(0, 240 + i) for i in range(60)], out, lse, 0, SCALE)
    s.pool.close()


@pytest.mark.parametrize("n,hkv", [(3000, 1), (9000, 2)])
def test_split_over_the_cache(cuda_lib, n, hkv):
    """The parts of a split join by references and log-sum-exps that are as large."""
    s = Setup(4 * hkv, hkv, 16, 1, n, seed=n)
    s.length = n
    s.fill(spread=2)
    q = bf16(s.rng.standard_normal((6, 4 * hkv, 128)) * powers(s.rng, (6, 4 * hkv, 1)))
    for i in range(6):
        one = q[i:i + 1].contiguous()
        out, lse = s.decode(one, [n])
        check(s, one, [(0, n - 1)], out, lse, 0, SCALE)
    out, lse = s.prefill(q, [6], [n])
    check(s, q, [(0, n - 6 + i) for i in range(6)], out, lse, 0, SCALE)
    s.pool.close()
