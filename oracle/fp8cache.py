"""The 8-bit cache in numpy, fp64: e4m3 codes with one power-of-two scale per
16 tokens, KV head and tensor; rotary positions; the append; attention under a
sliding window with first tokens kept.

Everything is written from the definitions in ``include/kvint2.h``; rounding to
e4m3 or bf16 happens once, from fp64, where the header says that it happens.
"""

import math

import numpy as np

TILE, D = 16, 128
E_MIN, E_MAX = -64, 7


# ---- e4m3 -------------------------------------------------------------------

def e4m3_table():
    """The 256 values: 4 exponent bits (bias 7), 3 mantissa bits, no infinities."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


TABLE = e4m3_table()


def e4m3_round(x):
    """Nearest e4m3 value, ties to even, saturated to +-448 (NaN stays)."""
    x = np.asarray(x, np.float64)
    mag = np.where(np.isfinite(x), np.abs(x), 448.0)
    _, ex = np.frexp(np.maximum(mag, 2.0 ** -6))
    step = np.ldexp(1.0, ex - 4)
    y = np.copysign(np.minimum(np.rint(mag / step) * step, 448.0), x)
    return np.where(np.isnan(x), np.nan, y)


def e4m3_encode(x):
    """Codes of e4m3 values (already rounded)."""
    x = np.asarray(x, np.float64)
    pos = TABLE[:127]
    c = np.searchsorted(pos, np.abs(np.where(np.isnan(x), 0.0, x))).astype(np.uint8)
    c = np.where(np.signbit(x), c | 128, c)
    return np.where(np.isnan(x), 127, c).astype(np.uint8)


# ---- stored order -----------------------------------------------------------

def places():
    """Byte offsets of (token, channel) in a tile's K and V codes: two int arrays [16, 128]."""
    t, c = np.meshgrid(np.arange(TILE), np.arange(D), indexing="ij")
    k = (t // 8) * 1024 + (c // 64) * 512 + (t % 8) * 64 + c % 64
    v = (t % 2 + 2 * (t // 8)) * 512 + (c // 16) * 64 + ((t % 8) // 2) * 16 + c % 16
    return k, v


class Cache:
    """codes uint8 [pages, Hkv, page_size/16, 2, 2048], exps int8 [pages, Hkv, page_size/16, 2]."""

    def __init__(self, num_pages, hkv, page_size):
        self.P, self.H, self.pages = page_size, hkv, num_pages
        shape = (num_pages, hkv, page_size // TILE, 2)
        self.codes = np.zeros((*shape, TILE * D), np.uint8)
        self.exps = np.zeros(shape, np.int8)

    def rows(self, table, n, h):
        """K and V [n, 128] of KV head h of the sequence with page ids `table`; rows of a
        bad page are absent: also returns which rows are present."""
        kv = np.zeros((2, n, D))
        ok = np.zeros(n, bool)
        place = places()
        for t0 in range(0, n, TILE):
            pid, sub = int(table[t0 // self.P]), t0 // TILE % (self.P // TILE)
            if not 0 <= pid < self.pages:
                continue
            m = min(TILE, n - t0)
            ok[t0:t0 + m] = True
            for w in range(2):
                x = TABLE[self.codes[pid, h, sub, w]] * 2.0 ** float(self.exps[pid, h, sub, w])
                kv[w, t0:t0 + m] = x[place[w]][:m]
        return kv[0], kv[1], ok


# ---- rotary positions -------------------------------------------------------

class Rope:
    def __init__(self, rotary_dim=0, style="half", theta=10000.0, scaling="none", factor=1.0,
                 original_max_position=0, beta_fast=0.0, beta_slow=0.0, attention_factor=0.0, inv_freq=None):
        d = self.rd = rotary_dim
        self.style = style
        i = np.arange(d // 2)
        att = attention_factor
        if inv_freq is not None:
            w = np.asarray(inv_freq, np.float64)
        else:
            base = theta * factor ** (d / (d - 2)) if scaling == "ntk" and d else theta
            w = base ** (-2.0 * i / d) if d else np.zeros(0)
            if scaling == "linear":
                w = w / factor
            elif scaling == "yarn" and d:
                def index(turns):
                    return d * math.log(original_max_position / (turns * 2 * math.pi)) / (2 * math.log(base))
                lo = max(math.floor(index(beta_fast or 32.0)), 0)
                hi = min(math.ceil(index(beta_slow or 1.0)), d - 1)
                keep = 1.0 - np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
                w = w * keep + w / factor * (1 - keep)
                att = att or 0.1 * math.log(factor) + 1.0
        self.w, self.att = w, float(np.float32(att or 1.0))

    def pairs(self):
        """Channel indexes of the first and second members of the rotated pairs."""
        n = self.rd // 2
        i = np.arange(n)
        return (i, i + n) if self.style == "half" else (2 * i, 2 * i + 1)

    def rotate(self, x, pos):
        """x [n, H, 128] at positions pos [n]."""
        x = np.array(x, np.float64)
        one, two = self.pairs()
        ang = np.asarray(pos, np.float64)[:, None] * self.w
        c, s = self.att * np.cos(ang)[:, None], self.att * np.sin(ang)[:, None]
        a, b = x[..., one].copy(), x[..., two].copy()
        x[..., one], x[..., two] = a * c - b * s, b * c + a * s
        return x

    def reach(self, x):
        """|a| + |b| of each channel's pair times att (|x| where not rotated): what an error in
        cos and sin is multiplied by."""
        x = np.abs(np.asarray(x, np.float64))
        y = x.copy()
        one, two = self.pairs()
        y[..., one] = y[..., two] = (x[..., one] + x[..., two]) * self.att
        return y

    def lengths(self, x):
        """Per row the largest pair length times att, or magnitude where not rotated."""
        x = np.asarray(x, np.float64)
        one, two = self.pairs()
        y = np.abs(x).copy()
        y[..., one] = y[..., two] = np.hypot(x[..., one], x[..., two]) * self.att
        return y.max(-1)


def exponent(m):
    """The smallest e with m <= 448 * 2^e, within the format's range."""
    if not m > 0:
        return E_MIN
    e = E_MIN
    while e < E_MAX and m > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(cache, rope, k, v, start, count, table):
    """Tokens k, v [T, H, 128] (fp64 of bf16 values) of all sequences in order.  Returns what
    the stored K and V would be before rounding, by place: a list of (index of the codes
    array, fp64 value / 2^e, slack of K's rotation / 2^e)."""
    place, wrote, row = places(), [], 0
    for s, (p0, n) in enumerate(zip(start, count)):
        p0, n = int(p0), int(n)
        pos = np.arange(p0, p0 + n)
        x = [rope.rotate(k[row:row + n], pos), np.asarray(v[row:row + n], np.float64)]
        slack = [rope.reach(k[row:row + n]) * 2.0 ** -21, np.zeros((n, cache.H, D))]
        size = [rope.lengths(k[row:row + n]), np.abs(x[1]).max(-1) if n else np.zeros((0, cache.H))]
        dead = [~np.isfinite(k[row:row + n]).all(-1), ~np.isfinite(v[row:row + n]).all(-1)]
        for tile in range(p0 // TILE, (p0 + n + TILE - 1) // TILE if n else p0 // TILE):
            lo, hi = max(p0, tile * TILE), min(p0 + n, tile * TILE + TILE)
            pid, sub = int(table[s][tile * TILE // cache.P]), tile % (cache.P // TILE)
            if not 0 <= pid < cache.pages:
                continue
            for h in range(cache.H):
                for w in range(2):
                    live = ~dead[w][lo - p0:hi - p0, h]
                    e = exponent(float(np.max(size[w][lo - p0:hi - p0, h][live], initial=0.0)))
                    codes = cache.codes[pid, h, sub, w]
                    first = lo - tile * TILE
                    if first:
                        old = int(cache.exps[pid, h, sub, w])
                        e = max(e, old)
                        at = place[w][:first].ravel()
                        if e > old:
                            codes[at] = e4m3_encode(e4m3_round(TABLE[codes[at]] * 2.0 ** (old - e)))
                    for t in range(lo, hi):
                        at = place[w][t - tile * TILE]
                        y = np.full(D, np.nan) if dead[w][t - p0, h] else x[w][t - p0, h] * 2.0 ** -e
                        codes[at] = e4m3_encode(e4m3_round(y))
                        wrote.append(((pid, h, sub, w, at), y, slack[w][t - p0, h] * 2.0 ** -e))
                    cache.exps[pid, h, sub, w] = e
        row += n
    return wrote


# ---- attention --------------------------------------------------------------

def visible(pos, n, window, n_sink):
    """Which of the first n cached tokens a query at `pos` sees."""
    j = np.arange(n)
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < n_sink)
    return see


def attend(q, k, v, see, scale):
    """q [128] over rows k, v [n, 128] where `see`; returns out [128], lse, and what the error
    bounds need: sum of p |v| and the largest scale * sum |q k|."""
    k, v = k[see], v[see]
    if not len(k):
        return np.zeros(D), -math.inf, np.zeros(D), 0.0
    with np.errstate(invalid="ignore"):
        x = k @ q * scale
        m = x.max()
        p = np.exp(x - m)
        l = p.sum()
        return p @ v / l, m + math.log(l), p @ np.abs(v) / l, float(np.max(np.abs(k) @ np.abs(q)) * abs(scale))
