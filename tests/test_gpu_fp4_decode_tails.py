"""Single-token attention over the 4-bit cache: small weights count whatever V's scales are."""

import math

import numpy as np
import pytest

from bit_kv_cache_12_gb300 import native
from oracle import fp4cache as f4
from oracle import fp8cache as fc
from tests.fp4_util import Setup
from tests.fp8_util import bf16, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [0x01, 0x08, 0x38, 0x7E])          # 2^-9, 2^-6, 1, 448
def test_decode_of_one_large_weight_before_many_small_ones(cuda_lib, byte):
    """One dominant token, and others whose weights of 2^-19.2 of it add up to a tenth of it, for every size of V's scales.
    More pairs than splits: a warp goes through 8192 tokens.  A large value takes the one, its negative all others.

    Bound: the output's rounding (2^-8 of it), a weight's to fp16 (2^-11 of each), exp2 (2^-21) and the logits' errors
    (2^-18 of scale * sum |q k|, and 2^-22), 1.01 for their products; the largest weight is at least
    2^7 and fp16's steps end at 2^-24: a token's weight is off by 2^-32 of the largest at most."""
    hkv, n, B = 8, 65536, 310
    s = Setup(hkv, hkv, 32, 1, n, seed=byte)
    s.pool.close()
    s.pool = native.KVPool(native.KV_POOL_FP4, 1, hkv, hkv, 32, s.pages, B)
    t = s.model.tiles
    t[..., :1024] = 0x00                                              # keys: zeros,
    t[..., 1024:2048] = 0xFF                                          # values -6,
    t[..., 2048:2176] = 0x38                                          # scales 1
    t[..., 2176:] = byte
    at, where = f4.places(), 5                                        # (before the others: the reference is its logit)
    tile = t[s.table[0][where // 32], :, where // 16 % 2]
    tile[:, at[0][where % 16]] = 0x22                                 # the dominant key: ones (two channels to a byte)
    v, shift = at[2][where % 16], at[3][where % 16]
    tile[:, v] = (tile[:, v] & (0xF0 >> shift)) | (0x7 << shift).astype(np.uint8)   # its values 6
    s.view = s.pool.fp4_view(0)
    s.upload()
    q = bf16(np.full((B, hkv, 128), 1.1796875))
    scale = 19.2 * math.log(2) / (128 * 1.1796875)
    table = np.repeat(s.table, B, 0)
    out, lse = s.decode(q, [n] * B, scale=scale, table=table)
    for b in (0, 17, B - 1):
        k, val, ok = s.model.rows(s.table[0], n, 3)
        ref, rl, av, sqk = fc.attend(f64(q)[b, 3], k, val, ok, scale)
        logit = 2.0 ** -18 * sqk + 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -20 + 2 * logit) * av * 1.01 + n * 2.0 ** -32 * np.abs(val).max()
        assert np.all(np.abs(out[b, 3] - ref) <= tol), (float(np.abs(out[b, 3] - ref).max()), float(tol.max()), float(ref[0]))
        assert abs(lse[b, 3] - rl) <= logit + 2.0 ** -20 + 2.0 ** -22 * abs(rl)
        for h in range(hkv):
            np.testing.assert_array_equal(out[b, h], out[0, 0])
    assert s.pool.error() == 0
    s.pool.close()
