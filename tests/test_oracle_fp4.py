"""Pins of the 4-bit cache's model to facts that do not come from it."""

import numpy as np
import pytest

from oracle import fp4cache as f4
from oracle import fp8cache as fc


def test_e2m1_by_hand():
    # value -> code, ties to the even mantissa, saturated
    cases = {0.0: 0, 0.25: 0, 0.26: 1, 0.5: 1, 0.74: 1, 0.75: 2, 1.0: 2, 1.25: 2, 1.3: 3, 1.75: 4, 2.0: 4, 2.5: 4, 2.6: 5,
             3.5: 6, 4.0: 6, 5.0: 6, 5.1: 7, 6.0: 7, 7.0: 7, 1e30: 7}
    for x, c in cases.items():
        assert f4.e2m1_encode(x) == c, x
        assert f4.e2m1_encode(-x) == c + 8, -x
    np.testing.assert_array_equal(f4.e2m1_encode(f4.E2M1), np.arange(16))
    # nearest, by brute force
    x = np.random.default_rng(0).uniform(-8, 8, 2000)
    best = np.abs(np.clip(x, -6, 6)[:, None] - f4.E2M1).min(1)
    np.testing.assert_allclose(np.abs(f4.E2M1[f4.e2m1_encode(x)] - np.clip(x, -6, 6)), best, atol=1e-15)


def test_stored_order():
    k, ksh, v, vsh, ks, vs = f4.places()
    for at, sh, lo in ((k, ksh, 0), (v, vsh, 1024)):
        slots = (2 * (at - lo) + sh // 4).ravel()
        assert sorted(slots) == list(range(2048))
    for at, lo in ((ks, 2048), (vs, 2176)):
        assert sorted(np.unique(at)) == list(range(lo, lo + 128))
        blocks = at.reshape(16, 8, 16)
        assert (blocks == blocks[:, :, :1]).all()
    # by hand: token 11, channel 77 = block 4, its channel 13
    assert k[11, 77] == 11 * 64 + 38 and ksh[11, 77] == 4
    assert v[11, 77] == 1024 + 512 + 64 * 6 + 16 * 1 + 0 + 2 + 1 and vsh[11, 77] == 4
    assert ks[11, 77] == 2048 + 92 and vs[11, 77] == 2176 + 32 + 16 + 2 + 1


@pytest.mark.parametrize("e", [0, -5, 9])
def test_quantize(e):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 128)) * 2.0 ** e * np.exp(rng.standard_normal((40, 1)))
    x = np.float32(x).view(np.uint32) & 0xFFFF0000
    x = x.view(np.float32).astype(np.float64)
    codes, scales = f4.quantize(x, e)
    s = fc.TABLE[scales] * 2.0 ** e
    y = (f4.E2M1[codes].reshape(40, 8, 16) * s[..., None])
    top = np.abs(x).reshape(40, 8, 16).max(-1)
    # the scale is a sixth of the largest within half a step of 4 bits; an error is at most half the largest step
    # (2 scales wide), or what is cut where the scale was rounded down
    assert (np.abs(s * 6 - top) <= top * 2.0 ** -4).all()
    err = np.abs(y - x.reshape(40, 8, 16))
    assert (err <= np.maximum(s, top - 6 * s)[..., None] + 1e-300).all()
    # values on the grid stay
    codes2, scales2 = f4.quantize(y.reshape(40, 128), e)
    full = (np.abs(f4.E2M1[codes]).reshape(40, 8, 16).max(-1) == 6)
    assert full.mean() > 0.5
    same = (f4.E2M1[codes2] * 1.0).reshape(40, 8, 16) * (fc.TABLE[scales2] * 2.0 ** e)[..., None]
    np.testing.assert_array_equal(same[full], y[full])


def test_quantize_edges():
    x = np.zeros((4, 128))
    x[0, :16] = 1e-5                      # below half the smallest scale times 6
    x[1, :16] = 1e9                       # beyond the range
    x[1, 16:32] = -1e9
    x[2, 5], x[2, 40] = np.nan, -np.inf
    codes, scales = f4.quantize(x, 0)
    assert scales[0, 0] == 0 and (codes[0] == 0).all()
    assert fc.TABLE[scales[1, 0]] == 448 and (codes[1, :16] == 7).all() and (codes[1, 16:32] == 15).all()
    assert np.isnan(fc.TABLE[scales[2, 0]]) and np.isnan(fc.TABLE[scales[2, 2]]) and scales[2, 1] == 0
    assert (scales[3] == 0).all()


@pytest.mark.parametrize("page", [16, 32])
def test_append_reads_back(page):
    rng = np.random.default_rng(page)
    c = f4.Cache(9, 2, page, 1, -2)
    c.tiles[...] = rng.integers(0, 126, c.tiles.shape)
    before = c.tiles.copy()
    table = rng.permutation(9)[:8].reshape(2, 4)
    k, v = rng.standard_normal((2, 25, 2, 128))
    c.append(k, v, [3, 30], [20, 5], table)
    for s, (lo, n, row) in enumerate(((3, 20, 0), (30, 5, 20))):
        for h in range(2):
            got = c.rows(table[s], lo + n, h)
            for w, x in enumerate((k, v)):
                codes, scales = f4.quantize(x[row:row + n, h], c.exp[w])
                want = f4.E2M1[codes].reshape(n, 8, 16) * fc.TABLE[scales][..., None] * 2.0 ** c.exp[w]
                np.testing.assert_array_equal(got[w][lo:], want.reshape(n, 128))
    # nothing else moved: writing the old values of the same slots back restores the bytes
    old = f4.Cache(9, 2, page, 1, -2)
    old.tiles[...] = before
    np.testing.assert_array_equal(old.rows(table[0], 3, 1)[1], c.rows(table[0], 3, 1)[1])
    untouched = np.setdiff1d(np.arange(9), table.ravel())
    np.testing.assert_array_equal(c.tiles[untouched], before[untouched])
    assert not c.rows([99, -1, 3, 4], 40, 0)[2][:min(40, 2 * page)].any()


def test_axes():
    rope = fc.Rope(rotary_dim=64, style="interleaved", theta=100.0)
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 2, 128))
    pos = rng.integers(0, 1000, (3, 5))
    # the same position on every axis is the plain rotation
    axis = [i % 3 for i in range(32)]
    np.testing.assert_allclose(f4.rotate_axes(rope, axis, x, np.stack([pos[0]] * 3)), rope.rotate(x, pos[0]), atol=1e-12)
    # each pair like the plain rotation by its own axis
    got = f4.rotate_axes(rope, axis, x, pos)
    for i in range(32):
        np.testing.assert_allclose(got[..., 2 * i:2 * i + 2], rope.rotate(x, pos[i % 3])[..., 2 * i:2 * i + 2], atol=1e-12)
    np.testing.assert_array_equal(got[..., 64:], x[..., 64:])
