"""Helpers of the 4-bit cache's tests: pools, stored state to and from the fp64 model, the
library calls, and the error bounds they are held to."""

import math

import numpy as np
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp4cache as f4
from oracle import fp8cache as fc
from tests.fp8_util import bf16, f64, i32


class Setup:
    """A pool, its fp64 model and the page table of sequences with up to `longest` tokens."""

    def __init__(self, hq=8, hkv=2, page=16, seqs=3, longest=64, k_exp=0, v_exp=0, layers=1, layer=0, seed=0, spare=2):
        self.hq, self.hkv, self.page, self.seqs, self.layer = hq, hkv, page, seqs, layer
        self.rng = np.random.default_rng(seed)
        self.width = max(1, -(-longest // page))
        self.pages = seqs * self.width + spare
        self.table = self.rng.permutation(self.pages)[:seqs * self.width].reshape(seqs, self.width).astype(np.int32)
        self.pool = native.KVPool(native.KV_POOL_FP4, layers, hq, hkv, page, self.pages, seqs)
        self.model = f4.Cache(self.pages, hkv, page, k_exp, v_exp)
        native.kv_pool_set_fp4_range(self.pool.handle, layer, k_exp, v_exp)
        self.view = self.pool.fp4_view(layer)

    def upload(self):
        self.view.copy_(torch.from_numpy(self.model.tiles))
        torch.cuda.synchronize()

    def fill(self, spread=0.2, middle=0.3):
        """Random codes and scales (no NaN), in the model and in the pool."""
        r, t = self.rng, self.model.tiles
        t[..., :2048] = r.integers(0, 256, (*t.shape[:-1], 2048))
        scale = middle * np.exp(spread * r.standard_normal((*t.shape[:-1], 256)))
        t[..., 2048:] = fc.e4m3_encode(fc.e4m3_round(scale))
        self.upload()

    def append(self, k, v, start, count, cu=None, most=None, table=None, stream=None):
        """kv_append_fp4 of bf16 device tensors [T, Hkv, 128] (any token stride)."""
        count = np.asarray(count)
        cu = np.concatenate([[0], np.cumsum(count)]) if cu is None else cu
        native.kv_append_fp4(self.pool.handle, self.layer, len(count), k, k.stride(0), v, v.stride(0), i32(cu), i32(start),
                             i32(self.table if table is None else table), self.width,
                             int(max(count.max(), 0)) if most is None else most, stream)
        torch.cuda.synchronize()

    def read(self, start, count, cu=None, most=None, table=None, rows=None, out=None):
        """kv_read_fp4: k and v, bf16 device tensors (7.0 where nothing was written)."""
        count = np.asarray(count)
        cu = np.concatenate([[0], np.cumsum(count)]) if cu is None else cu
        rows = int(cu[-1]) if rows is None else rows
        if out is None:
            out = torch.full((2, rows, self.hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        native.kv_read_fp4(self.pool.handle, self.layer, len(count), i32(cu), i32(start),
                           i32(self.table if table is None else table), self.width,
                           int(max(count.max(), 0)) if most is None else most, out[0], out[0].stride(0), out[1],
                           out[1].stride(0))
        torch.cuda.synchronize()
        return out

    def check_tiles(self):
        np.testing.assert_array_equal(self.view.cpu().numpy(), self.model.tiles)

    def decode(self, q, n, window=0, sinks=0, scale=1 / math.sqrt(128), max_len=None, table=None, stream=None):
        B = len(n)
        max_len = int(max(max(n), 0)) if max_len is None else max_len
        bytes_ = native.kv_decode_workspace_bytes(self.pool.handle, B, max_len)
        ws = torch.full((bytes_ + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((B, self.hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, self.hq), float("nan"), device="cuda")
        native.kv_decode_attention_fp4(self.pool.handle, self.layer, B, q, i32(n),
                                       i32(self.table if table is None else table), self.width, max_len, scale, window,
                                       sinks, out, lse, ws, bytes_, stream)
        torch.cuda.synchronize()
        return f64(out), f64(lse)

    def check_rows(self, q, rows, out, lse, window, sinks, scale=1 / math.sqrt(128), table=None, lens=None):
        """Every (row, head) of out / lse against the fp64 model; rows: (sequence, position)."""
        table = self.table if table is None else table
        G = self.hq // self.hkv
        q, cached = f64(q), {}
        for i, (s, pos) in enumerate(rows):
            n = int(lens[s])
            for h in range(self.hq):
                if (s, h // G) not in cached:
                    cached[(s, h // G)] = self.model.rows(table[s], n, h // G)
                k, v, ok = cached[(s, h // G)]
                see = fc.visible(pos, n, window, sinks) & ok
                check_row(out[i, h], lse[i, h], q[i, h], k, v, see, scale, (i, h, s, pos), 2.0 ** self.model.exp[1])


def check_row(out, lse, q, k, v, see, scale, what, unit):
    """One output row of the single-token attention against fp64; unit: 2^e of V.

    Bound of the output: its own rounding (bf16, 2^-8 relative, as of everything below half a
    step); a weight is rounded to fp16 and once more times V's scale (2^-11 each) and has its
    exp2's error (2^-21); the error of a logit moves a weight by as much: 128 products summed
    in fp32, each partial sum off by at most 2^-22 of scale * sum |q k| (two bits more than
    fp32's half step, for the tensor cores' accumulation), 9 partial sums, the scaling to base
    2 and the difference to the reference (2^-23 each): 2^-18 in all.  The largest weight is
    at least 2^3, and fp16's steps end at 2^-24: a weight is off by at most 2^-25 (2^-28 of the
    largest), and the product with V's scale by 2^-25 again, times a code of at most 6."""
    ref, rl, av, sqk = fc.attend(q, k, v, see, scale)
    if not see.any():
        assert np.all(out == 0) and lse == -math.inf, what
        return
    if np.isnan(rl):
        assert np.isnan(out).all() and np.isnan(lse), what
        return
    logit = 2.0 ** -18 * sqk + 2.0 ** -22
    drop = see.sum() * 2.0 ** -28 * (np.nanmax(np.abs(v[see])) + 6 * unit)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -20 + 2 * logit) * av * 1.01 + drop + 1e-38
    live = ~np.isnan(ref)
    assert np.array_equal(np.isnan(out), ~live), what
    over = np.abs(out - ref)[live] - tol[live]
    assert np.all(over <= 0), (what, float(over.max()), float(np.abs(out - ref)[live].max()))
    assert abs(lse - rl) <= logit + 2.0 ** -20 + 2.0 ** -22 * abs(rl), (what, lse, rl)
