"""The fp64 model of the 8-bit cache, pinned to facts from outside it."""

import math

import numpy as np
import pytest
import torch

from oracle import fp8cache as fc


def test_e4m3_values_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(fc.TABLE, codes.view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 100, rng.standard_normal(4000) * 0.01,
                        (fc.TABLE[:126] + fc.TABLE[1:127]) / 2, [0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(fc.e4m3_round(x), want.double().numpy())
    np.testing.assert_array_equal(fc.e4m3_encode(fc.e4m3_round(x)), want.view(torch.uint8).numpy())
    assert fc.e4m3_round(1e9) == 448 and fc.e4m3_round(-np.inf) == -448 and np.isnan(fc.e4m3_round(np.nan))


def test_stored_order_is_a_permutation():
    for p in fc.places():
        assert sorted(p.ravel()) == list(range(2048))


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [0, 32, 64, 96, 128])
def test_rotation_keeps_lengths_and_relative_positions(style, rd):
    rng = np.random.default_rng(1)
    r = fc.Rope(rd, style, theta=1e4)
    x, y = rng.standard_normal((2, 1, 3, 128))
    a = r.rotate(x, [5])
    np.testing.assert_allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    np.testing.assert_array_equal(a[..., rd:], x[..., rd:])
    # the product depends on the distance alone
    d = [(r.rotate(x, [p + 7]) * r.rotate(y, [p])).sum(-1) for p in (0, 100, 99999)]
    np.testing.assert_allclose(d[1], d[0], rtol=1e-9, atol=1e-9)
    np.testing.assert_allclose(d[2], d[0], rtol=1e-8, atol=1e-8)


def test_speeds_of_the_scalings():
    base = fc.Rope(128, theta=1e4).w
    assert base[0] == 1 and base[63] == pytest.approx(1e4 ** (-126 / 128))
    np.testing.assert_allclose(fc.Rope(128, theta=1e4, scaling="linear", factor=4).w, base / 4)
    ntk = fc.Rope(128, theta=1e4, scaling="ntk", factor=4).w
    assert ntk[0] == 1 and ntk[63] == pytest.approx(base[63] / 4)        # the slowest pair is stretched by the factor
    y = fc.Rope(128, theta=1e4, scaling="yarn", factor=4, original_max_position=4096)
    turns = 4096 * base / (2 * math.pi)
    np.testing.assert_allclose(y.w[turns > 40], base[turns > 40])
    np.testing.assert_allclose(y.w[turns < 0.8], base[turns < 0.8] / 4)
    assert np.all(np.diff(y.w / base) <= 1e-12)
    assert y.att == pytest.approx(1 + 0.1 * math.log(4), rel=1e-6)


def test_exponent_borders():
    assert fc.exponent(0.0) == -64 and fc.exponent(448.0) == 0 and fc.exponent(np.nextafter(448.0, 500)) == 1
    assert fc.exponent(7.0) == -6 and fc.exponent(1e9) == 7 and fc.exponent(1e-30) == -64


def test_append_in_pieces_keeps_values_within_a_step():
    rng = np.random.default_rng(2)
    n, H = 37, 2
    k, v = rng.standard_normal((2, n, H, 128)) * np.array([1.0, 30.0])[None, None, :, None]
    rope = fc.Rope(128)
    for cuts in ([37], [1] * 37, [5, 20, 12]):
        cache, at = fc.Cache(4, H, 16), 0
        table = np.array([[2, 0, 3]])
        for c in cuts:
            fc.append(cache, rope, k[at:at + c], v[at:at + c], [at], [c], table)
            at += c
        for h in range(H):
            kk, vv, ok = cache.rows(table[0], n, h)
            assert ok.all()
            # two roundings at most matter: to the code, and to a subnormal when the tile's scale grew
            for got, want in ((kk, rope.rotate(k, np.arange(n))[:, h]), (vv, v[:, h])):
                scale = 2.0 ** np.repeat(cache.exps[table[0][:3], h, 0, 0 if got is kk else 1].astype(float), 16)[:n]
                assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2 * 2.0 ** -9 * scale[:, None])


def test_attention_against_brute_force():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal(128), rng.standard_normal((40, 128)), rng.standard_normal((40, 128))
    see = fc.visible(30, 40, 8, 3)
    assert list(np.flatnonzero(see)) == [0, 1, 2] + list(range(23, 31))
    assert fc.visible(30, 40, 0, 3).sum() == 31 and not fc.visible(-1, 40, 8, 3).any()
    out, lse, _, _ = fc.attend(q, k, v, see, 0.1)
    w = [math.exp(0.1 * float(q @ k[j])) for j in np.flatnonzero(see)]
    np.testing.assert_allclose(out, sum(a * v[j] for a, j in zip(w, np.flatnonzero(see))) / sum(w), rtol=1e-12)
    assert lse == pytest.approx(math.log(sum(w)))
    assert fc.attend(q, k, v, np.zeros(40, bool), 0.1)[1] == -math.inf
