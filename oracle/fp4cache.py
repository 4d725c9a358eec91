"""The 4-bit cache in numpy, fp64: e2m1 codes with one e4m3 scale per token, KV head,
tensor and block of 16 channels; rotary positions with several axes; attention over
packed rows.

Everything is written from the definitions in ``include/kvint2.h``.
"""

import numpy as np

from . import fp8cache as fc

TILE, D, BLOCK = 16, 128, 16
TILE_BYTES = 2304

# 2 exponent bits (bias 1), 1 mantissa bit, then the sign
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def e2m1_encode(x):
    """Codes of the nearest e2m1 values, ties to even mantissa, saturated to +-6."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 6.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    a = np.rint(a / step) * step
    return (np.searchsorted(E2M1[:8], a) + np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def places():
    """Of (token, channel) in a tile: byte and bit shift of the K code and of the V code,
    bytes of the two scales; six int arrays [16, 128]."""
    t, c = np.meshgrid(np.arange(TILE), np.arange(D), indexing="ij")
    k = 64 * t + c // 2
    v = 1024 + 512 * (c // 64) + 64 * (c % 16 // 2) + 16 * (t % 8 // 2) + 4 * (c // 16 % 4) + 2 * (t // 8) + c % 2
    ks = 2048 + 8 * t + c // 16
    vs = 2176 + 32 * (t % 8 // 2) + 4 * (c // 16) + 2 * (t // 8) + t % 2
    return k, 4 * (c % 2), v, 4 * (t % 2), ks, vs


def quantize(x, e):
    """Rows [..., 128] (fp64 of bf16 values) -> codes uint8 [..., 128] and e4m3 scale bytes [..., 8]."""
    y = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], D // BLOCK, BLOCK) * 2.0 ** -e
    dead = ~np.isfinite(y).all(-1)
    y = np.where(dead[..., None], 0.0, y)
    s = fc.e4m3_round(np.abs(y).max(-1) / 6.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, y / s[..., None], 0.0)
    codes = e2m1_encode(q)
    return codes.reshape(np.shape(x)), np.where(dead, 0x7F, fc.e4m3_encode(s)).astype(np.uint8)


class Cache:
    """tiles uint8 [pages, Hkv, page_size/16, 2304]; k_exp, v_exp: the layer's exponents."""

    def __init__(self, num_pages, hkv, page_size, k_exp=0, v_exp=0):
        self.P, self.H, self.pages = page_size, hkv, num_pages
        self.exp = (k_exp, v_exp)
        self.tiles = np.zeros((num_pages, hkv, page_size // TILE, TILE_BYTES), np.uint8)

    def values(self, tiles):
        """K and V [..., 16, 128] of stored tiles [..., 2304]."""
        k, ksh, v, vsh, ks, vs = places()
        return [E2M1[(tiles[..., at] >> sh) & 15] * fc.TABLE[tiles[..., sc]] * 2.0 ** e
                for at, sh, sc, e in ((k, ksh, ks, self.exp[0]), (v, vsh, vs, self.exp[1]))]

    def rows(self, table, n, h):
        """K and V [n, 128] of KV head h of the sequence with page ids `table`; rows of a bad
        page are absent: also returns which rows are present."""
        tiles = -(-n // TILE)
        at = np.arange(tiles) * TILE
        pid, sub = np.asarray(table)[at // self.P].astype(np.int64), at // TILE % (self.P // TILE)
        good = (pid >= 0) & (pid < self.pages)
        kv = self.values(self.tiles[np.where(good, pid, 0), h, sub])
        ok = np.repeat(good, TILE)[:n]
        return (*[np.where(ok[:, None], x.reshape(-1, D)[:n], 0.0) for x in kv], ok)

    def append(self, k, v, start, count, table):
        """Rows k, v [T, H, 128] of all sequences in order."""
        at = places()
        new = [quantize(x, e) for x, e in zip((k, v), self.exp)]
        row = 0
        for s, (p0, n) in enumerate(zip(start, count)):
            for i in range(int(n)):
                pos = int(p0) + i
                pid, sub, t = int(table[s][pos // self.P]), pos // TILE % (self.P // TILE), pos % TILE
                if not 0 <= pid < self.pages:
                    continue
                for h in range(self.H):
                    tile = self.tiles[pid, h, sub]
                    for w in range(2):
                        codes, scales = new[w][0][row + i, h], new[w][1][row + i, h]
                        byte, shift = at[2 * w][t], at[2 * w + 1][t]
                        for half in (0, 4):        # (two channels of a K byte)
                            m = shift == half
                            tile[byte[m]] = (tile[byte[m]] & (0xF0 >> half)) | (codes[m] << half)
                        tile[at[4 + w][t][::BLOCK]] = scales
            row += int(n)


def rotate_axes(rope, axis, x, pos):
    """x [n, H, 128]; pair i turns by pos[axis[i]] [n] (``fp8cache.Rope``)."""
    x = np.array(x, np.float64)
    one, two = rope.pairs()
    ang = np.stack([np.asarray(pos[a], np.float64) for a in axis], 1) * rope.w
    c, s = rope.att * np.cos(ang)[:, None], rope.att * np.sin(ang)[:, None]
    a, b = x[..., one].copy(), x[..., two].copy()
    x[..., one], x[..., two] = a * c - b * s, b * c + a * s
    return x
