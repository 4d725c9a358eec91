"""Helpers of the 8-bit cache tests: pools, stored state to and from the fp64
model, the library calls, and the error bounds they are held to."""

import math

import numpy as np
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc


def bf16(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


class Setup:
    """A pool, its fp64 model and the page table of sequences with up to `longest` tokens."""

    def __init__(self, hq=8, hkv=2, page=16, seqs=3, longest=64, rope=None, layers=1, layer=0, seed=0, spare=2):
        self.hq, self.hkv, self.page, self.seqs, self.layer = hq, hkv, page, seqs, layer
        self.rng = np.random.default_rng(seed)
        self.width = max(1, -(-longest // page))
        self.pages = seqs * self.width + spare
        self.table = self.rng.permutation(self.pages)[:seqs * self.width].reshape(seqs, self.width).astype(np.int32)
        self.pool = native.KVPool(native.KV_POOL_FP8, layers, hq, hkv, page, self.pages, seqs)
        self.model = fc.Cache(self.pages, hkv, page)
        self.rope = fc.Rope(**(rope or {}))
        if rope:
            native.kv_pool_set_rope(self.pool.handle, layer, native.rope_config(**rope))
        self.codes, self.exps = self.pool.fp8_views(layer)

    def upload(self):
        self.codes.copy_(torch.from_numpy(self.model.codes))
        self.exps.copy_(torch.from_numpy(self.model.exps))
        torch.cuda.synchronize()

    def fill(self, spread=1):
        """Random stored codes (no NaN) and exponents, in the model and in the pool."""
        r = self.rng
        x = np.clip(r.standard_normal(self.model.codes.shape) * 100, -448, 448)
        self.model.codes[...] = fc.e4m3_encode(fc.e4m3_round(x))
        self.model.exps[...] = r.integers(-7 - spread, -7 + spread + 1, self.model.exps.shape)
        self.upload()

    def append(self, q, k, v, start, count, cu=None, most=None, q_out=None, table=None, stream=None, pool=None):
        """kv_append_fp8 of bf16 device tensors q (or None), k, v [T, heads, 128] (any token stride)."""
        count = np.asarray(count)
        if cu is None:
            cu = np.concatenate([[0], np.cumsum(count)])
        if q is not None and q_out is None:
            q_out = torch.full((q.shape[0], self.hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        native.kv_append_fp8((pool or self.pool).handle, self.layer, len(count), q, 0 if q is None else q.stride(0), k,
                             k.stride(0), v, v.stride(0), i32(cu), i32(start),
                             i32(self.table if table is None else table), self.width,
                             int(max(count.max(), 0)) if most is None else most, q_out, stream)
        torch.cuda.synchronize()
        return q_out

    def decode(self, q, n, window=0, sinks=0, scale=1 / math.sqrt(128), max_len=None, table=None, stream=None):
        B = len(n)
        max_len = int(max(max(n), 0)) if max_len is None else max_len
        bytes_ = native.kv_decode_workspace_bytes(self.pool.handle, B, max_len)
        ws = torch.full((bytes_ + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((B, self.hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, self.hq), float("nan"), device="cuda")
        native.kv_decode_attention_fp8(self.pool.handle, self.layer, B, q, i32(n),
                                       i32(self.table if table is None else table), self.width, max_len, scale, window,
                                       sinks, out, lse, ws, bytes_, stream)
        torch.cuda.synchronize()
        return f64(out), f64(lse)

    def prefill(self, q, count, n, window=0, sinks=0, scale=1 / math.sqrt(128), most=None, max_len=None, table=None,
                cu=None, out=None, lse=None):
        count = np.asarray(count)
        cu = np.concatenate([[0], np.cumsum(count)]) if cu is None else cu
        most = int(max(count)) if most is None else most
        max_len = int(max(max(n), 0)) if max_len is None else max_len
        bytes_ = native.kv_prefill_workspace_bytes(self.pool.handle, len(count), most, max_len)
        assert bytes_ > 0
        ws = torch.full((bytes_ + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((q.shape[0], self.hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
        lse = torch.full((q.shape[0], self.hq), float("nan"), device="cuda") if lse is None else lse
        native.kv_prefill_attention_fp8(self.pool.handle, self.layer, len(count), q, i32(cu), i32(n),
                                        i32(self.table if table is None else table), self.width, most, max_len, scale,
                                        window, sinks, out, lse, ws, bytes_)
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
                check_row(out[i, h], lse[i, h], q[i, h], k, v, see, scale, (i, h, s, pos))


def check_row(out, lse, q, k, v, see, scale, what):
    """One output row against fp64.

    Bound of the output: its own rounding (bf16, 2^-8); the weights' rounding to fp16 for the
    product with V (2^-11 of each) and their exp2 (2^-21); the error of a logit, which moves a
    weight by as much: 128 products summed in fp32, each partial sum off by at most 2^-22 of
    scale * sum |q k| (two bits more than fp32's half step, for the tensor cores' accumulation),
    8 or 16 partial sums, the scaling to base 2 and the difference to the reference (2^-23 each):
    2^-18 in all; weights under fp16's range (2^-30 of the largest) dropped."""
    ref, rl, av, sqk = fc.attend(q, k, v, see, scale)
    if not see.any():
        assert np.all(out == 0) and lse == -math.inf, what
        return
    if np.isnan(rl):
        assert np.isnan(out).all() and np.isnan(lse), what
        return
    logit = 2.0 ** -18 * sqk + 2.0 ** -22
    drop = see.sum() * 2.0 ** -30 * np.max(np.abs(v[see]))
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -20 + 2 * logit) * av * 1.01 + drop + 1e-38
    live = ~np.isnan(ref)
    assert np.array_equal(np.isnan(out), ~live), what
    over = np.abs(out - ref)[live] - tol[live]
    assert np.all(over <= 0), (what, float(over.max()), float(np.abs(out - ref)[live].max()))
    assert abs(lse - rl) <= logit + 2.0 ** -20 + 2.0 ** -22 * abs(rl), (what, lse, rl)


def check_codes(s, wrote):
    """The pool's stored state against the model after `fc.append` returned `wrote`: exponents
    and codes that came from elsewhere equal, new codes the rounding of a value within the
    rotation's slack (half a step where the model's value is a tie)."""
    codes, exps = s.codes.cpu().numpy(), s.exps.cpu().numpy()
    np.testing.assert_array_equal(exps, s.model.exps)
    loose = np.zeros(codes.shape, bool)
    for (p, h, t, w, at), y, slack in wrote:
        got = fc.TABLE[codes[p, h, t, w][at]]
        if np.isnan(y).any():
            assert np.isnan(got).all()
        else:
            assert np.all(got >= fc.e4m3_round(y - slack)) and np.all(got <= fc.e4m3_round(y + slack)), (p, h, t, w)
        loose[p, h, t, w][at] = True
    a, b = fc.TABLE[codes], fc.TABLE[s.model.codes]
    same = (a == b) | (np.isnan(a) & np.isnan(b))
    assert np.all(same | loose)
    # later steps start from what the pool holds
    s.model.codes[...] = codes


def check_rotated(got, x, rope, pos):
    """bf16 rows against the rotation in fp64: the rounding of a value within 2^-21 of |a| + |b|."""
    y, slack = rope.rotate(x, pos), rope.reach(x) * 2.0 ** -21
    lo = f64(torch.as_tensor(y - slack).to(torch.bfloat16))
    hi = f64(torch.as_tensor(y + slack).to(torch.bfloat16))
    # torch rounds fp64 to bf16 by way of fp32: a step of slack covers the double rounding
    lo, hi = lo - np.abs(lo) * 2.0 ** -23, hi + np.abs(hi) * 2.0 ** -23
    assert np.all((got >= lo) & (got <= hi)), float(np.max(np.maximum(lo - got, got - hi)))
