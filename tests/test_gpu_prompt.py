"""Causal attention over packed bf16 rows, against fp64."""

import math

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc
from tests.fp8_util import bf16, f64, i32

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)


class Prompt:
    """Packed rows and a call; q, k, v are parts of wider rows."""

    def __init__(self, hq=8, hkv=2, count=(5,), keys=(5,), seed=0, kind=native.KV_POOL_BF16, size=1.0, spare=0):
        self.rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.count, self.keys = hq, hkv, list(count), list(keys)
        self.cq, self.ck = (np.concatenate([[0], np.cumsum(x)]) for x in (count, keys))
        self.pool = native.KVPool(kind, 1, hq, hkv, 16, 1, max(1, len(count)))
        self.tq, self.tk = int(self.cq[-1]) + spare, max(1, int(self.ck[-1]) + spare)
        self.qw = bf16(self.rng.standard_normal((self.tq, hq + 1, 128)) * size)
        self.kw = bf16(self.rng.standard_normal((self.tk, 2 * hkv + 1, 128)))
        self.q, self.k, self.v = self.qw[:, 1:], self.kw[:, :hkv], self.kw[:, hkv + 1:]

    def run(self, window=0, sinks=0, scale=SCALE, most=None, longest=None, lse=True, stream=None, cq=None, ck=None, q_rows=None,
            kv_rows=None):
        most = max(self.count) if most is None else most
        longest = max(self.keys) if longest is None else longest
        n = len(self.count)
        wb = native.kv_prompt_workspace_bytes(self.pool.handle, n, most, longest)
        assert wb > 0
        ws = torch.full((wb,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((self.tq, self.hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full((self.tq, self.hq), 7.0, device="cuda")
        native.kv_prompt_attention(self.pool.handle, n, self.q, self.q.stride(0), self.tq if q_rows is None else q_rows, self.k,
                                   self.k.stride(0), self.v, self.v.stride(0), self.tk if kv_rows is None else kv_rows,
                                   i32(self.cq if cq is None else cq), i32(self.ck if ck is None else ck), most, longest, scale,
                                   window, sinks, out, l if lse else None, ws, wb, stream)
        torch.cuda.synchronize()
        return f64(out), f64(l)

    def check(self, out, lse, window=0, sinks=0, scale=SCALE, sample=None, seqs=None):
        rows = [(b, i) for b, c in enumerate(self.count) for i in range(c) if seqs is None or b in seqs]
        if sample is not None and sample < len(rows):
            last = len(rows) - 1
            rows = [rows[i] for i in sorted({0, last, *self.rng.choice(len(rows), sample, replace=False).tolist()})]
        q, k, v = f64(self.q), f64(self.k), f64(self.v)
        G = self.hq // self.hkv
        for b, i in rows:
            n, at = self.keys[b], int(self.cq[b]) + i
            pos = n - self.count[b] + i
            see = fc.visible(pos, n, window, sinks)
            part = slice(int(self.ck[b]), int(self.ck[b]) + n)
            for h in range(self.hq):
                check_row(out[at, h], lse[at, h], q[at, h], k[part, h // G], v[part, h // G], see, scale, (b, i, h))

    def close(self):
        assert self.pool.error() == 0
        self.pool.close()


def check_row(out, lse, q, k, v, see, scale, what):
    """One row against fp64.  Bound of the output: its own rounding (bf16, 2^-8 relative, as of
    everything below half a step), the weights' rounding to bf16 for the product with V (2^-8 of
    each), their exp2 (2^-21), and the error of a logit, which moves a weight by as much: 128
    products summed in fp32, each of at most 16 partial sums off by 2^-22 of scale * sum |q k|,
    scaled to base 2 and taken from the reference (2^-23 each): 2^-18 in all.  Weights are never
    below fp32's normal range while they count."""
    with np.errstate(invalid="ignore", over="ignore"):
        ref, rl, av, sqk = fc.attend(q, k, v, see, scale)
    if not see.any():
        assert np.all(out == 0) and lse == -math.inf, what
        return
    if np.isnan(rl):
        assert np.isnan(out).all() and np.isnan(lse), what
        return
    logit = 2.0 ** -18 * sqk + 2.0 ** -22
    live = np.isfinite(v[see]).all(0)
    assert np.array_equal(np.isfinite(out), live), what
    drop = see.sum() * 2.0 ** -100 * np.max(np.abs(v[see][:, live]), initial=0.0)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -20 + 2 * logit) * av * 1.01 + drop + 1e-38
    off = np.abs(out[live] - ref[live])
    over = off - tol[live]
    assert np.all(over <= 0), (what, float(over.max()), float(off.max()))
    assert abs(lse - rl) <= logit + 2.0 ** -20 + 2.0 ** -22 * abs(rl), (what, lse, rl)


RAGGED = [1, 0, 17, 64, 130, 5, 300], [1, 30, 17, 100, 400, 3, 301]       # the sixth: more queries than keys


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2), (5, 5)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 5), (200, 70)])
def test_ragged(cuda_lib, hq, hkv, window, sinks):
    p = Prompt(hq, hkv, *RAGGED, seed=hq)
    p.check(*p.run(window, sinks), window, sinks, sample=150)
    p.close()


@pytest.mark.parametrize("count,keys,window,sinks,hkv", [
    ([3], [9000], 0, 0, 1), ([3], [9000], 4096, 64, 2), ([700, 1], [5000, 2500], 0, 0, 2), ([1100], [1100], 0, 0, 1),
    ([600], [6001], 513, 130, 1), ([40, 300], [3000, 2000], 300, 20, 4), ([1], [1], 0, 0, 1), ([257], [257], 0, 0, 8)])
def test_long(cuda_lib, count, keys, window, sinks, hkv):
    p = Prompt(4 * hkv, hkv, count, keys, seed=keys[0])
    p.check(*p.run(window, sinks), window, sinks, sample=40)
    p.close()


def test_many_sequences(cuda_lib):
    rng = np.random.default_rng(3)
    count = rng.integers(0, 90, 200)
    p = Prompt(8, 2, count, count, seed=4)
    p.check(*p.run(), sample=200)
    p.close()


@pytest.mark.parametrize("n", [100, 1000])
def test_scales(cuda_lib, n):
    """Large and small queries, negative and zero softmax scales, logits that rise along the keys."""
    p = Prompt(4, 1, [50], [n], seed=n)
    p.q.mul_(torch.tensor([1e-3, 1.0, 30.0, 1e4], device="cuda")[:, None].to(torch.bfloat16))
    for scale in (SCALE, -0.3, 0.0, 1e-30):
        p.check(*p.run(scale=scale), scale=scale)
    p.q[:, [0, 1, 2, 3]] = 1.0
    p.k[...] = (torch.arange(n, device="cuda") * 100 / n)[:, None, None].to(torch.bfloat16)
    for scale in (0.5, -0.5):
        p.check(*p.run(scale=scale), scale=scale)
    p.close()


@pytest.mark.parametrize("size", [1e4, 1e8, 1e30])
def test_large_logits(cuda_lib, size):
    """Logits whose fp32 steps are larger than one: a mean of the values, and the one of the largest logit where no
    other is near."""
    p = Prompt(8, 1, [70], [200], seed=5, size=size)
    out, lse = p.run()
    q, k, v = f64(p.q), f64(p.k)[:, 0], f64(p.v)[:, 0]
    for i in range(70):
        n = 131 + i
        for h in range(8):
            x = k[:n] @ q[i, h] * SCALE
            error = 2.0 ** -17 * (np.abs(k[:n]) @ np.abs(q[i, h])).max() * SCALE + 2.0 ** -20
            order = np.argsort(x)[::-1]
            near = v[:n][x >= x[order[0]] - 2 * error - 60]
            slack = 2.0 ** -7 * np.abs(near).max(0) + 1e-12
            assert (out[i, h] >= near.min(0) - slack).all() and (out[i, h] <= near.max(0) + slack).all()
            if x[order[0]] - x[order[1]] > 2 * error + 60:
                np.testing.assert_array_equal(out[i, h], v[order[0]])
            assert abs(lse[i, h] - x[order[0]]) <= error + 10
    p.close()


@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 4), (150, 100)])
def test_what_is_hidden_stays_hidden(cuda_lib, window, sinks):
    """NaN and infinities in keys and values that no query, or not this query, sees."""
    p = Prompt(8, 2, [150, 40, 3, 200], [333, 40, 3, 200], seed=window, spare=9)
    want = p.run(window, sinks)
    p.check(*want, window, sinks, sample=100)
    bad = [float("nan"), float("inf"), -float("inf")]
    ck = p.ck
    # keys and values behind the last sequence, and of sequence 0 before its window
    p.k[ck[4]:] = bad[0]
    p.v[ck[4]:] = bad[1]
    if window:
        low = 333 - 150 - window + 1
        p.k[sinks:low], p.v[sinks:low] = bad[0], bad[2]
    got = p.run(window, sinks)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    # single places: rows that see them are not finite there, all others as before
    p.v[ck[0] + 250, 0, 17], p.v[ck[0] + 251, 1, 0], p.v[ck[0] + 300, 0, 99] = bad
    p.v[ck[3] + 7, 1, 64], p.v[ck[3] + 130, 0, 127] = bad[1], bad[0]
    p.v[ck[1] + 39, 0, 3] = bad[2]
    out, lse = p.run(window, sinks)
    p.check(out, lse, window, sinks)
    hit = np.zeros(out.shape, bool)
    for b, key, g, c in ((0, 250, 0, 17), (0, 251, 1, 0), (0, 300, 0, 99), (3, 7, 1, 64), (3, 130, 0, 127), (1, 39, 0, 3)):
        for i in range(p.count[b]):
            if fc.visible(p.keys[b] - p.count[b] + i, p.keys[b], window, sinks)[key]:
                hit[int(p.cq[b]) + i, 4 * g:4 * g + 4, c] = True
    np.testing.assert_array_equal(out[~hit], want[0][~hit])
    assert not np.isfinite(out[hit]).any()
    np.testing.assert_array_equal(lse, want[1])
    # a key: the whole row
    p.k[ck[3] + 100, 1, 5] = bad[0]
    out, lse = p.run(window, sinks)
    p.check(out, lse, window, sinks)
    # a query: its own row
    p.q[int(p.cq[1]) + 11, 2, 9] = bad[0]
    out2, lse2 = p.run(window, sinks)
    assert np.isnan(out2[int(p.cq[1]) + 11, 2]).all() and np.isnan(lse2[int(p.cq[1]) + 11, 2])
    out2[int(p.cq[1]) + 11, 2], lse2[int(p.cq[1]) + 11, 2] = out[int(p.cq[1]) + 11, 2], lse[int(p.cq[1]) + 11, 2]
    np.testing.assert_array_equal(out2, out)
    np.testing.assert_array_equal(lse2, lse)
    p.close()


def test_ranges(cuda_lib):
    """Sequences above their bounds or outside the rows are left out; rows behind the last one are not touched."""
    p = Prompt(8, 2, [20, 33, 7, 12], [40, 33, 20, 12], seed=8, spare=5)
    want = p.run()
    p.check(*want)
    assert (want[0][p.cq[4]:] == 7).all() and (want[1][p.cq[4]:] == 7).all()

    def left_out(lost, **kw):
        out, lse = p.run(**kw)
        assert p.pool.error() == 3, kw
        for b in range(4):
            part = slice(int(p.cq[b]), int(p.cq[b + 1]))
            if b in lost:
                assert (out[part] == 7).all() and (lse[part] == 7).all(), (kw, b)
            else:
                np.testing.assert_array_equal(out[part], want[0][part])
                np.testing.assert_array_equal(lse[part], want[1][part])
    left_out([1], most=32)
    left_out([0], longest=39)
    left_out([3], q_rows=int(p.cq[4]) - 1)
    left_out([2, 3], kv_rows=int(p.ck[3]) - 1)
    left_out([0], cq=[-1, *p.cq[1:]])
    left_out([0], ck=[-2, *p.ck[1:]])
    bad = p.cq.copy()
    bad[1] = 60                                     # the first is too long, the second falls
    left_out([0, 1], cq=bad)
    p.close()


def test_repeats_streams_graph_and_workspace(cuda_lib):
    """The same bits on a second call, another stream, without lse, with a larger workspace's bounds, and replayed from
    graphs with other lengths; pools of every kind."""
    p = Prompt(8, 2, [30, 2], [2000, 700], seed=6)
    first = p.run()
    p.check(*first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (p.run(), p.run(stream=side)):
        np.testing.assert_array_equal(got[0], first[0])
        np.testing.assert_array_equal(got[1], first[1])
    np.testing.assert_array_equal(p.run(lse=False)[0], first[0])
    p.check(*p.run(most=500, longest=5000))
    wb = native.kv_prompt_workspace_bytes(p.pool.handle, 2, 30, 2000)
    for s, mq, mk in ((1, 30, 2000), (2, 1, 2000), (2, 30, 1), (1, 1, 1), (2, 16, 1000)):
        assert native.kv_prompt_workspace_bytes(p.pool.handle, s, mq, mk) <= wb
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    cq, ck = i32(p.cq), i32(p.ck)
    out = torch.empty(p.tq, 8, 128, dtype=torch.bfloat16, device="cuda")

    def call(n, window):
        native.kv_prompt_attention(p.pool.handle, n, p.q, p.q.stride(0), p.tq, p.k, p.k.stride(0), p.v, p.v.stride(0), p.tk, cq,
                                   ck, 30, 2000, SCALE, window, 0, out, None, ws, wb)
    call(2, 0)
    graphs = []
    for args in ((2, 0), (1, 50)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*args)
        graphs.append((g, args))
    for count, keys in (([30, 2], [2000, 700]), ([7, 25], [7, 1999]), ([0, 30], [100, 30])):
        p.count, p.keys = count, keys
        p.cq, p.ck = (np.concatenate([[0], np.cumsum(x)]) for x in (count, keys))
        cq.copy_(i32(p.cq))
        ck.copy_(i32(p.ck))
        for g, (n, window) in graphs:
            g.replay()
            torch.cuda.synchronize()
            got = f64(out)
            p.count, p.keys = count[:n], keys[:n]
            want = p.run(window, most=30, longest=2000, cq=p.cq[:n + 1], ck=p.ck[:n + 1])
            rows = int(p.cq[n])
            np.testing.assert_array_equal(got[:rows], want[0][:rows])
            p.check(*want, window, seqs=range(n), sample=20)
            p.count, p.keys = count, keys
    p.close()
    outs = []
    for kind in (0, 1, 2, 4):
        x = Prompt(8, 2, [30, 2], [200, 70], seed=6, kind=kind)
        outs.append(x.run())
        x.close()
    for o in outs[1:]:
        np.testing.assert_array_equal(o[0], outs[0][0])


@pytest.mark.parametrize("count,keys", [([300, 100], [600, 100]), ([40], [3000])])
def test_wait_that_runs_out(cuda_lib, count, keys):
    """Values that are never handed over: the call ends and reports it, the rows that were lost are not numbers, the
    others stand, and the next call is right.  The second case splits the keys."""
    p = Prompt(8, 2, count, keys, seed=12, kind=native.KV_POOL_FP4)
    want = p.run()
    native.kv_debug_stall_first_copy(p.pool.handle, True, 2000)
    out, lse = p.run()
    assert p.pool.error() == 4
    lost = np.isnan(out).any(-1)
    assert lost.any() and (~lost).any() and np.isnan(out[lost]).all()
    np.testing.assert_array_equal(out[~lost], want[0][~lost])
    native.kv_debug_stall_first_copy(p.pool.handle, False)
    again = p.run()
    np.testing.assert_array_equal(again[0], want[0])
    np.testing.assert_array_equal(again[1], want[1])
    p.close()
