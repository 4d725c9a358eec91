"""Single-token attention over the 4-bit cache, against the fp64 model."""

import math

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp4cache as f4
from oracle import fp8cache as fc
from tests.fp4_util import Setup
from tests.fp8_util import bf16, f64, i32

pytestmark = pytest.mark.gpu


def decode_and_check(s, q, n, window=0, sinks=0, scale=1 / math.sqrt(128), **kw):
    out, lse = s.decode(q, n, window, sinks, scale, **kw)
    s.check_rows(q, [(b, m - 1) for b, m in enumerate(n)], out, lse, window, sinks, scale, lens=n)
    return out, lse


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 5), (128, 64), (1000, 16)])
def test_decode(cuda_lib, hq, hkv, page, window, sinks):
    n = [0, 1, 15, 16, 17, 31, 33, 100, 129, 500, 1023]
    s = Setup(hq, hkv, page, len(n), 1024, 1, -2, seed=hq + page)
    s.fill()
    decode_and_check(s, bf16(s.rng.standard_normal((len(n), hq, 128))), n, window, sinks)
    assert s.pool.error() == 0
    s.pool.close()


@pytest.mark.parametrize("n,window,sinks,hkv", [(9000, 0, 0, 1), (9000, 4096, 64, 2), (20001, 0, 0, 8), (20001, 7777, 33, 1)])
def test_decode_long(cuda_lib, n, window, sinks, hkv):
    """One long sequence beside a short one: the split over the cache and its joining."""
    s = Setup(4 * hkv, hkv, 16, 2, n, seed=n)
    s.fill()
    decode_and_check(s, bf16(s.rng.standard_normal((2, 4 * hkv, 128))), [n, 40], window, sinks)
    s.pool.close()


def test_decode_of_many_sequences(cuda_lib):
    s = Setup(8, 2, 16, 150, 300, seed=5)
    s.fill()
    n = s.rng.integers(0, 301, 150)
    decode_and_check(s, bf16(s.rng.standard_normal((150, 8, 128))), n.tolist(), max_len=300)
    s.pool.close()


@pytest.mark.parametrize("n", [40, 300, 3000])
def test_decode_scales(cuda_lib, n):
    """Wide spreads of scales up to the largest, tiny ones, large and small queries, negative and zero
    softmax scales, steep softmax, logits that rise along the cache."""
    s = Setup(4, 1, 16, 2, n, seed=n)
    s.fill(spread=2.5)
    q = bf16(s.rng.standard_normal((2, 4, 128)) * np.array([1e-3, 1.0, 30.0, 1e4])[None, :, None])
    decode_and_check(s, q, [n, n // 2])
    decode_and_check(s, q[:, [2, 2, 0, 1]].contiguous(), [n, n // 2], scale=-0.3)
    decode_and_check(s, q, [n, n // 2], scale=0.0)
    unit = bf16(s.rng.standard_normal((2, 4, 128)))
    for byte in (0, 1, 0x7E):              # V's scales: zero, the smallest, the largest
        s.model.tiles[..., 2176:] = byte
        s.upload()
        decode_and_check(s, unit, [n, n // 2])
    for e in ((-32, 32), (32, -32)):
        s.model.exp = e
        native.kv_pool_set_fp4_range(s.pool.handle, 0, *e)
        decode_and_check(s, unit, [n, n // 2], scale=2.0 ** (-4 - e[0]))
    s.pool.close()
    # the reference moves all the way
    s = Setup(4, 1, 16, 2, n, seed=n)
    s.fill()
    rise = np.repeat((np.arange(n) + 1.0)[:, None] * 100 / n, 128, 1)[:, None]
    s.model.append(rise, s.rng.standard_normal((n, 1, 128)), [0], [n], s.table)
    s.upload()
    decode_and_check(s, bf16(np.full((2, 4, 128), 1.0)), [n, n // 2], scale=0.5)
    s.pool.close()


@pytest.mark.parametrize("size", [1e5, 1e8, 1e30])
def test_decode_large_logits(cuda_lib, size):
    """Logits whose fp32 steps are larger than one: the largest weight stays in range."""
    s = Setup(8, 1, 16, 1, 400, seed=7)
    s.fill()
    s.model.tiles[..., 2176:] = fc.e4m3_encode(448.0)
    s.upload()
    q = bf16(s.rng.standard_normal((1, 8, 128)) * size)
    out, lse = s.decode(q, [400])
    k, v, _ = s.model.rows(s.table[0], 400, 0)
    x = (k @ f64(q)[0].T) / math.sqrt(128)
    for h in range(8):
        # tokens whose logits lie within the roundings of the largest may win
        near = x[:, h] >= x[:, h].max() - 2.0 ** -17 * np.abs(k).sum(1) * np.abs(f64(q)[0, h]).max() - 40
        lo, hi = v[near].min(0), v[near].max(0)
        assert np.isfinite(out[0, h]).all() and (out[0, h] >= lo - 2.0 ** -7 * np.abs(lo) - 1e-6).all()
        assert (out[0, h] <= hi + 2.0 ** -7 * np.abs(hi) + 1e-6).all()
        assert abs(lse[0, h] - x[:, h].max()) <= 2.0 ** -17 * (np.abs(k) @ np.abs(f64(q)[0, h])).max() + 10
    s.pool.close()


@pytest.mark.parametrize("page", [16, 32])
def test_decode_hides_what_it_should(cuda_lib, page):
    """NaN scales behind the end, before the window and in pages with a bad id do not reach the output;
    in a visible token they do."""
    s = Setup(8, 2, page, 3, 200, seed=page)
    s.fill()
    q = bf16(s.rng.standard_normal((3, 8, 128)))
    clean = s.model.tiles.copy()
    n, window, sinks = [150, 77, 199], 50, 9
    want = decode_and_check(s, q, n, window, sinks)
    _, _, _, _, ks, vs = f4.places()
    for b in range(3):
        for j in range(s.width * page):
            if j < n[b] and (j >= n[b] - window or j < sinks):
                continue
            p, sub = s.table[b][j // page], j // 16 % (page // 16)
            s.model.tiles[p, :, sub][:, np.concatenate([ks[j % 16], vs[j % 16]])] = 0x7F
    s.upload()
    got = s.decode(q, n, window, sinks)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    s.model.tiles[...] = clean
    s.upload()
    table = s.table.copy()
    table[0, 1], table[1, -1], table[2, 2] = -1, s.pages + 5, s.pages
    out, lse = s.decode(q, n, table=table)
    s.check_rows(q, [(b, m - 1) for b, m in enumerate(n)], out, lse, 0, 0, lens=n, table=table)
    assert s.pool.error() == 1
    s.model.tiles[s.table[0][3 * 16 // page], 1, 3 * 16 // 16 % (page // 16), vs[2, 30]] = 0xFF   # one block of V
    s.model.tiles[s.table[1][0], 0, 0, ks[4, 100]] = 0x7F
    s.upload()
    out, _ = decode_and_check(s, q, n)
    assert np.isnan(out[0, 4:, 16:32]).all() and np.isfinite(out[0, :4]).all() and np.isfinite(out[0, 4:, 32:]).all()
    s.pool.close()


def test_decode_lengths_out_of_range(cuda_lib):
    s = Setup(8, 2, 16, 3, 128, seed=1)
    s.fill()
    q = bf16(s.rng.standard_normal((3, 8, 128)))
    out, lse = s.decode(q, [500, -3, 60], max_len=100)
    s.check_rows(q, [(0, 99), (1, -1), (2, 59)], out, lse, 0, 0, lens=[100, 0, 60])
    assert s.pool.error() == 2 and s.pool.error() == 0
    # a query that is not finite is not a number; the others stand
    q[0, 1, 5], q[0, 2, 6] = float("nan"), float("inf")
    out, lse = s.decode(q, [100, 20, 60])
    assert np.isnan(out[0, 1:3]).all() and np.isnan(lse[0, 1:3]).all()
    keep = [0, 3, 4, 5, 6, 7]
    assert np.isfinite(out[0, keep]).all() and np.isfinite(out[1:]).all()
    # all-zero queries weigh all tokens alike
    out, lse = s.decode(torch.zeros_like(q), [100, 20, 60])
    s.check_rows(torch.zeros_like(q), [(0, 99), (1, 19), (2, 59)], out, lse, 0, 0, lens=[100, 20, 60])
    s.pool.close()


def test_decode_repeats_streams_and_graph(cuda_lib):
    """The same bits on a second call, on another stream, and replayed from a graph with other lengths;
    lse may be left out; one workspace serves smaller calls; two graphs share it."""
    s = Setup(8, 2, 16, 2, 5000, seed=2)
    s.fill()
    q = bf16(s.rng.standard_normal((2, 8, 128)))
    first = s.decode(q, [5000, 321])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (s.decode(q, [5000, 321]), s.decode(q, [5000, 321], stream=side)):
        np.testing.assert_array_equal(got[0], first[0])
        np.testing.assert_array_equal(got[1], first[1])
    n, table = i32([5000, 321]), i32(s.table)
    wb = native.kv_decode_workspace_bytes(s.pool.handle, 2, 5000)
    assert wb >= native.kv_decode_workspace_bytes(s.pool.handle, 1, 5000)
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda b=2: native.kv_decode_attention_fp4(s.pool.handle, 0, b, q, n, table, s.width, 5000,  # noqa: E731
                                                      1 / math.sqrt(128), 0, 0, out, None, ws, wb)
    call()
    call(1)
    graphs = []
    for b in (2, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(b)
        graphs.append(g)
    for lens in ([17, 4321], [5000, 321], [0, 1]):
        n.copy_(i32(lens))
        for g, b in zip(graphs, (2, 1)):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(f64(out)[:b], s.decode(q[:b], lens[:b], max_len=5000)[0])
    s.pool.close()


def test_decode_wait_that_runs_out(cuda_lib):
    """A copy that is never started: the call ends, reports it, and the next call is right."""
    s = Setup(8, 2, 16, 2, 3000, seed=9)
    s.fill()
    q = bf16(s.rng.standard_normal((2, 8, 128)))
    for n in ([3000, 17], [200, 17]):
        want = s.decode(q, n)
        native.kv_debug_stall_first_copy(s.pool.handle, True, 200)
        s.decode(q, n)
        assert s.pool.error() == 4
        native.kv_debug_stall_first_copy(s.pool.handle, False)
        got = s.decode(q, n)
        np.testing.assert_array_equal(got[0], want[0])
        assert s.pool.error() == 0
    s.pool.close()
