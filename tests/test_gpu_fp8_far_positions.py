"""Rotary angles far out: the 64-bit fractions of a turn against exact arithmetic, and the rotation of
rows and of appended tokens at positions beyond the first thousands."""

import math

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc
from tests.fp8_util import Setup, bf16, check_codes, check_rotated, f64, i32

pytestmark = pytest.mark.gpu

BITS = 256


def two_pi():
    """2 pi * 2^BITS as an integer (Machin: pi / 4 = 4 atan(1/5) - atan(1/239))."""
    def atan(n):
        one = (1 << (BITS + 32)) // n
        total, k = one, 1
        while one:
            one //= n * n
            total += (-1) ** k * (one // (2 * k + 1))
            k += 1
        return total
    return (8 * (4 * atan(5) - atan(239))) >> 32


TWO_PI = two_pi()


def quarter_offset(p, w):
    """p * w (w a double, taken exactly) in radians from its nearest quarter turn, and that quarter's number modulo 4."""
    num, den = float(w).as_integer_ratio()
    angle = (p * num << BITS) // den                       # radians * 2^BITS
    quarters = (4 * angle + TWO_PI // 2) // TWO_PI
    rest = 4 * angle - quarters * TWO_PI                   # 4 * offset * 2^BITS
    return math.ldexp(rest >> (BITS - 60), -62), quarters % 4


def test_two_pi():
    assert math.ldexp(TWO_PI >> (BITS - 60), -60) == pytest.approx(2 * math.pi, rel=1e-15)
    off, q = quarter_offset(1, math.pi / 2)
    assert abs(off + 6.123233995736766e-17) < 1e-18 and q == 1   # a double below pi / 2 by cos(it)


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("size", [1e-4, 0.05, 0.9, 40.0, -0.7])
@pytest.mark.parametrize("p", [1 << 20, (1 << 26) + 3, (1 << 31) - 2])
def test_angles_are_exact(cuda_lib, style, size, p):
    """Speeds that bring position p next to a quarter turn, where the small member of the rotated pair (1, 0) is
    the angle's distance from it.  The kernel's angle: the speed's fraction of a turn, off by 2^-64, times p
    <= 2^31, cut to 2^-34 of a turn, then relative errors (fp32 2^-24, sincospif 2^-22): 2^-32 of a turn, 2^-29
    radians, and bf16's 2^-8."""
    rng = np.random.default_rng(p & 0xFFFF)
    speeds, want = [], []
    while len(speeds) < 16:
        w = size * rng.uniform(0.5, 1)
        quarter = math.pi / 2
        w = (round(p * w / quarter) * quarter + rng.uniform(-1, 1) * 2.0 ** -18) / p
        off, q = quarter_offset(p, w)
        if 2.0 ** -22 < abs(off) < 2.0 ** -15:
            speeds.append(w)
            c, s = math.cos(off), math.sin(off)
            want.append([(c, s), (-s, c), (-c, -s), (s, -c)][q])
    pool = native.KVPool(native.KV_POOL_FP8, 1, 1, 1, 16, 1, 1)
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(rotary_dim=32, style=style, inv_freq=speeds))
    one, two = fc.Rope(32, style, inv_freq=speeds).pairs()
    x = np.zeros((1, 1, 128))
    x[0, 0, one] = 1.0
    q, out = bf16(x), torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    native.kv_rope_apply(pool.handle, 0, 1, i32([p]), q, 128, None, 0, out, 128, None, 0)
    got, want = f64(out)[0, 0], np.array(want)
    for member, channels in ((0, one), (1, two)):
        ref = want[:, member]
        assert np.all(np.abs(got[channels] - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref) + 2.0 ** -29)
    pool.close()
