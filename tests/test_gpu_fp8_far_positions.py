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


YARN = dict(scaling="yarn", factor=4.0, original_max_position=32768)
ROPES = [dict(rotary_dim=128, style="half", theta=1e6), dict(rotary_dim=96, style="half", theta=1e4, scaling="ntk", factor=8.0),
         dict(rotary_dim=64, style="interleaved", scaling="linear", factor=2.0), dict(rotary_dim=32, style="half"),
         dict(rotary_dim=128, style="interleaved", theta=5e5, **YARN)]


@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("n", [16, 33, 200])
@pytest.mark.parametrize("lo,hi", [(1, 1000), (1000, 131072), (131072, 1 << 24)])
def test_rows_at_far_positions(cuda_lib, rope, n, lo, hi):
    """Positions of every size, all rows on their own; up to 2^24 the model's own angle (position times speed in
    fp64) is off by 2^-28 radians at most, far below the 2^-21 that the check allows."""
    s = Setup(hq=8, hkv=2, rope=rope)
    pos = s.rng.integers(lo, hi, n)
    q, k = bf16(s.rng.standard_normal((n, 8, 128))), bf16(s.rng.standard_normal((n, 2, 128)))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    native.kv_rope_apply(s.pool.handle, 0, n, i32(pos), q, 1024, k, 256, qo, 1024, ko, 256)
    torch.cuda.synchronize()
    check_rotated(f64(qo), f64(q), s.rope, pos)
    check_rotated(f64(ko), f64(k), s.rope, pos)
    if rope["rotary_dim"] == 128:                              # and the check would see a row rotated by one position less
        with pytest.raises(AssertionError):
            check_rotated(f64(qo), f64(q), s.rope, pos - 1)
    s.pool.close()


@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("page", [16, 32])
def test_appends_at_far_positions(cuda_lib, rope, page):
    """Tokens that continue sequences of up to 10^6 tokens: codes, exponents and rotated q against the model."""
    start = np.array([0, 4099, 131071, 999983])
    s = Setup(hq=4, hkv=2, page=page, seqs=4, longest=160, rope=rope, seed=page)
    held, s.width = s.table, -(-(999983 + 200) // page)
    s.table = np.full((4, s.width), -1, np.int32)              # of the earlier pages the append needs none
    for b in range(4):
        first = start[b] // page
        room = min(held.shape[1], s.width - first)
        s.table[b, first:first + room] = held[b, :room]
    s.fill()
    for count in ([40, 1, 33, 17], [1, 70, 1, 2]):
        q, k, v = (bf16(s.rng.standard_normal((sum(count), h, 128))) for h in (4, 2, 2))
        qo = s.append(q, k, v, start, count)
        check_codes(s, fc.append(s.model, s.rope, f64(k), f64(v), start, count, s.table))
        check_rotated(f64(qo), f64(q), s.rope, np.concatenate([np.arange(a, a + c) for a, c in zip(start, count)]))
        start = start + count
    assert s.pool.error() == 0
    s.pool.close()


def test_rotated_rows_through_the_bf16_cache(cuda_lib):
    """kv_rope_apply in front of kv_append_bf16 and its decode, against fp64 on the rows that it wrote, at two places
    of the sequence; a query rotated to another position does not pass."""
    rng = np.random.default_rng(0)
    rope = dict(rotary_dim=128, theta=1e4)
    pool = native.KVPool(native.KV_POOL_BF16, 1, 4, 2, 16, 8, 2)
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(**rope))
    n = 50
    k, v = (bf16(np.tile(rng.standard_normal((n, 2, 128)), (2, 1, 1))) for _ in range(2))
    pos = np.r_[0:n, 1000:1000 + n]
    kr = torch.empty_like(k)
    native.kv_rope_apply(pool.handle, 0, 2 * n, i32(pos), None, 0, k, 256, None, 0, kr, 256)
    check_rotated(f64(kr), f64(k), fc.Rope(**rope), pos)
    pt = i32(np.arange(8).reshape(2, 4))
    native.kv_append_bf16(pool.handle, 0, 2, kr, v, i32([0, n, 2 * n]), i32([0, 0]), pt, 4, n)
    raw = bf16(np.tile(rng.standard_normal((1, 4, 128)), (2, 1, 1)))
    wb = native.kv_decode_workspace_bytes(pool.handle, 2, n)
    ws = torch.empty(max(16, wb), dtype=torch.uint8, device="cuda")

    def decode(at):
        q = raw.clone()
        native.kv_rope_apply(pool.handle, 0, 2, i32(at), q, 512, None, 0, q, 512, None, 0)
        out = torch.empty(2, 4, 128, device="cuda")
        native.kv_decode_attention_bf16(pool.handle, 0, 2, q, i32([n, n]), pt, 4, n, 0.05, out, ws, wb)
        torch.cuda.synchronize()
        return f64(q), f64(out)

    def off(q, out, b):
        """The largest excess over the error bound: weights of 16 bits, logits and sums in fp32 (2^-18 of sum |q k|)."""
        worst = -1.0
        for h in range(4):
            rows, values = f64(kr)[b * n:(b + 1) * n, h // 2], f64(v)[b * n:(b + 1) * n, h // 2]
            ref, _, mean, sqk = fc.attend(q[b, h], rows, values, np.ones(n, bool), 0.05)
            bound = (2.0 ** -15 + 2 * 2.0 ** -18 * sqk) * mean + 2.0 ** -20
            worst = max(worst, float(np.max(np.abs(out[b, h] - ref) - bound)))
        return worst

    q, out = decode([n - 1, 1000 + n - 1])
    check_rotated(q, f64(raw), fc.Rope(**rope), np.array([n - 1, 1000 + n - 1]))
    assert off(q, out, 0) <= 0 and off(q, out, 1) <= 0
    wrong = decode([0, 1000 + n - 1])[1]
    assert off(q, wrong, 0) > 0.01 and off(q, wrong, 1) <= 0
    pool.close()
