"""Single-token and prompt attention over the 8-bit cache, against the fp64 model."""

import math

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc
from tests.fp8_util import Setup, bf16, check_codes, f64, i32

pytestmark = pytest.mark.gpu


def decode_and_check(s, q, n, window=0, sinks=0, scale=1 / math.sqrt(128), **kw):
    out, lse = s.decode(q, n, window, sinks, scale, **kw)
    s.check_rows(q, [(b, m - 1) for b, m in enumerate(n)], out, lse, window, sinks, scale, lens=n)
    return out, lse


def prefill_and_check(s, q, count, n, window=0, sinks=0, scale=1 / math.sqrt(128), sample=None, **kw):
    out, lse = s.prefill(q, count, n, window, sinks, scale, **kw)
    rows = [(b, n[b] - c + i) for b, c in enumerate(count) for i in range(c)]
    pick = range(len(rows)) if sample is None else sorted(s.rng.choice(len(rows), min(sample, len(rows)), replace=False))
    pick = list(pick)
    s.check_rows(q[pick], [rows[i] for i in pick], out[pick], lse[pick], window, sinks, scale, lens=n)
    return out, lse


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 5), (128, 64), (1000, 16)])
def test_decode(cuda_lib, hq, hkv, page, window, sinks):
    n = [0, 1, 15, 16, 17, 31, 33, 100, 129, 500, 1023]
    s = Setup(hq, hkv, page, len(n), 1024, seed=hq + page)
    s.fill()
    decode_and_check(s, bf16(s.rng.standard_normal((len(n), hq, 128)) * 2), n, window, sinks)
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
    """Wide spreads of exponents, large and small queries, negative and zero softmax scales, steep softmax."""
    s = Setup(4, 1, 16, 2, n, seed=n)
    s.fill(spread=6)
    q = bf16(s.rng.standard_normal((2, 4, 128)) * np.array([1e-3, 1.0, 30.0, 1e4])[None, :, None])
    decode_and_check(s, q, [n, n // 2])
    decode_and_check(s, q[:, [2, 2, 0, 1]].contiguous(), [n, n // 2], scale=-0.3)
    decode_and_check(s, q, [n, n // 2], scale=0.0)
    s.model.exps[..., 0] = -7
    for e in (-64, 7):
        s.model.exps[..., 1] = e
        s.upload()
        decode_and_check(s, bf16(s.rng.standard_normal((2, 4, 128))), [n, n // 2])
    s.model.exps[..., 1] = s.rng.integers(-64, 8, s.model.exps.shape[:-1])
    s.upload()
    decode_and_check(s, bf16(s.rng.standard_normal((2, 4, 128))), [n, n // 2])
    # logits that rise along the cache: the reference moves all the way
    s.model.exps[...] = -7
    k_at, _ = fc.places()
    for j in range(n):
        p, t = s.table[0][j // 16], j % 16
        s.model.codes[p, 0, 0, 0][k_at[t]] = fc.e4m3_encode(fc.e4m3_round(np.full(128, 300.0 * (j + 1) / n)))
    s.upload()
    decode_and_check(s, bf16(np.full((2, 4, 128), 1.0)), [n, n // 2], scale=0.5)
    s.pool.close()


@pytest.mark.parametrize("page", [16, 32])
def test_decode_hides_what_it_should(cuda_lib, page):
    """NaN codes behind the end, before the window and in pages with a bad id do not reach the output;
    in a visible row they do."""
    s = Setup(8, 2, page, 3, 200, seed=page)
    s.fill()
    q = bf16(s.rng.standard_normal((3, 8, 128)))
    clean = s.model.codes.copy()
    n, window, sinks = [150, 77, 199], 50, 9
    want = decode_and_check(s, q, n, window, sinks)
    place = fc.places()
    for b in range(3):
        for j in range(s.width * page):
            if j < n[b] and (j >= n[b] - window or j < sinks):
                continue
            p, sub = s.table[b][j // page], j // 16 % (page // 16)
            for w in range(2):
                s.model.codes[p, :, sub, w][:, place[w][j % 16]] = 0x7F
    s.upload()
    got = s.decode(q, n, window, sinks)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    s.model.codes[...] = clean
    s.upload()
    table = s.table.copy()
    table[0, 1], table[1, -1], table[2, 2] = -1, s.pages + 5, s.pages
    out, lse = s.decode(q, n, table=table)
    s.check_rows(q, [(b, m - 1) for b, m in enumerate(n)], out, lse, 0, 0, lens=n, table=table)
    assert s.pool.error() == 1
    s.model.codes[s.table[0][3 * 16 // page], 1, 3 * 16 // 16 % (page // 16), 1][place[1][2]] = 0xFF
    s.model.codes[s.table[1][0], 0, 0, 0][place[0][4]] = 0x7F
    s.upload()
    decode_and_check(s, q, n)
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
    s.pool.close()


def test_decode_repeats_streams_and_graph(cuda_lib):
    """The same bits on a second call, on another stream, and replayed from a graph with other lengths;
    lse may be left out."""
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
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: native.kv_decode_attention_fp8(s.pool.handle, 0, 2, q, n, table, s.width, 5000,  # noqa: E731
                                                  1 / math.sqrt(128), 0, 0, out, None, ws, wb)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([17, 4321], [5000, 321], [0, 1]):
        n.copy_(i32(lens))
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(f64(out), s.decode(q, lens, max_len=5000)[0])
    s.pool.close()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 5), (200, 70)])
def test_prefill_ragged(cuda_lib, hq, hkv, page, window, sinks):
    count, n = [1, 0, 17, 64, 130, 5, 300], [1, 30, 17, 100, 400, 3, 301]       # the sixth: more queries than tokens
    s = Setup(hq, hkv, page, len(n), 416, seed=hq + page)
    s.fill()
    q = bf16(s.rng.standard_normal((sum(count), hq, 128)) * 2)
    prefill_and_check(s, q, count, n, window, sinks, sample=150)
    assert s.pool.error() == 0
    s.pool.close()


@pytest.mark.parametrize("count,n,window,sinks,hkv", [([3], [9000], 0, 0, 1), ([3], [9000], 4096, 64, 2),
                                                     ([700, 1], [5000, 2500], 0, 0, 2), ([1100], [1100], 0, 0, 1),
                                                     ([600], [6001], 513, 130, 1), ([40, 300], [3000, 2000], 300, 20, 4)])
def test_prefill_long(cuda_lib, count, n, window, sinks, hkv):
    s = Setup(4 * hkv, hkv, 16, len(n), max(n), seed=n[0])
    s.fill()
    q = bf16(s.rng.standard_normal((sum(count), 4 * hkv, 128)))
    prefill_and_check(s, q, count, n, window, sinks, sample=40)
    s.pool.close()


@pytest.mark.parametrize("n", [100, 1000])
def test_prefill_scales(cuda_lib, n):
    s = Setup(4, 1, 16, 1, n, seed=n)
    s.fill(spread=6)
    q = bf16(s.rng.standard_normal((50, 4, 128)) * np.array([1e-3, 1.0, 30.0, 1e4])[None, :, None])
    prefill_and_check(s, q, [50], [n])
    prefill_and_check(s, q[:, [2, 2, 0, 1]].contiguous(), [50], [n], scale=-0.3)
    prefill_and_check(s, q, [50], [n], scale=0.0)
    s.model.exps[..., 0] = -7
    for e in (-64, 7):
        s.model.exps[..., 1] = e
        s.upload()
        prefill_and_check(s, bf16(s.rng.standard_normal((50, 4, 128))), [50], [n])
    s.model.exps[...] = -7
    k_at, _ = fc.places()
    for j in range(n):
        p, t = s.table[0][j // 16], j % 16
        s.model.codes[p, 0, 0, 0][k_at[t]] = fc.e4m3_encode(fc.e4m3_round(np.full(128, 300.0 * (j + 1) / n)))
    s.upload()
    prefill_and_check(s, bf16(np.full((50, 4, 128), 1.0)), [50], [n], scale=0.5)
    s.pool.close()


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 9)])
def test_prefill_hides_what_it_should(cuda_lib, page, window, sinks):
    """A row of NaN in the cache reaches the queries that see it and no other; so do bad pages; what lies
    behind the end reaches none."""
    count, n = [90, 150], [200, 150]
    s = Setup(8, 2, page, 2, 256, seed=page)
    s.fill()
    q = bf16(s.rng.standard_normal((240, 8, 128)))
    place = fc.places()
    for b in range(2):
        for j in [130, 141, 7] + list(range(n[b], s.width * page)):
            p, sub = s.table[b][j // page], j // 16 % (page // 16)
            w = 0 if j == 141 else 1
            s.model.codes[p, b, sub, w][place[w][j % 16]] = 0x7F
    s.upload()
    out, lse = prefill_and_check(s, q, count, n, window, sinks)
    assert np.isnan(out).any() and np.isfinite(out[:, 4:][:90]).all()
    s.fill()
    table = s.table.copy()
    table[0, 1], table[1, 2] = -1, s.pages
    out, lse = s.prefill(q, count, n, window, sinks, table=table)
    rows = [(b, n[b] - c + i) for b, c in enumerate(count) for i in range(c)]
    s.check_rows(q, rows, out, lse, window, sinks, lens=n, table=table)
    assert s.pool.error() == 1
    s.pool.close()


def test_prefill_errors_and_rows_left_alone(cuda_lib):
    s = Setup(8, 2, 16, 3, 128, seed=1)
    s.fill()
    q = bf16(s.rng.standard_normal((100, 8, 128)))
    # the second has more queries than the host said; rows behind the last sequence are nobody's
    out, lse = s.prefill(q, [30, 40, 20], [100, 100, 500], most=30, max_len=120)
    rows = [(0, 70 + i) for i in range(30)] + [(2, 100 + i) for i in range(20)]
    at = np.r_[0:30, 70:90]
    s.check_rows(q[at.tolist()], rows, out[at], lse[at], 0, 0, lens=[100, 100, 120])
    assert np.isnan(out[30:70]).all() and np.isnan(out[90:]).all() and np.isnan(lse[30:70]).all() and np.isnan(lse[90:]).all()
    assert s.pool.error() in (2, 3)
    # a falling prefix sum (its rows would be the first sequence's too, which is over the bound)
    out, lse = s.prefill(q, [30, 0, 20], [100, -5, 100], cu=[0, 30, 20, 40], most=25)
    s.check_rows(q[20:40], [(2, 80 + i) for i in range(20)], out[20:40], lse[20:40], 0, 0, lens=[100, 0, 100])
    assert np.isnan(out[:20]).all() and np.isnan(out[40:]).all()
    s.pool.close()


def test_prefill_repeats_and_graph(cuda_lib):
    s = Setup(8, 2, 16, 2, 3000, seed=2)
    s.fill()
    q = bf16(s.rng.standard_normal((70, 8, 128)))
    first = s.prefill(q, [50, 20], [3000, 200])
    again = s.prefill(q, [50, 20], [3000, 200])
    np.testing.assert_array_equal(again[0], first[0])
    np.testing.assert_array_equal(again[1], first[1])
    cu, n, table = i32([0, 50, 70]), i32([3000, 200]), i32(s.table)
    wb = native.kv_prefill_workspace_bytes(s.pool.handle, 2, 50, 3000)
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    out = torch.empty(70, 8, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: native.kv_prefill_attention_fp8(s.pool.handle, 0, 2, q, cu, n, table, s.width, 50, 3000,  # noqa: E731
                                                   1 / math.sqrt(128), 0, 0, out, None, ws, wb)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens, c in (([100, 2999], [0, 20, 70]), ([3000, 200], [0, 50, 70])):
        n.copy_(i32(lens))
        cu.copy_(i32(c))
        out.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        want = s.prefill(q, np.diff(c), lens, most=50, max_len=3000)
        np.testing.assert_array_equal(f64(out), want[0])
    s.pool.close()


@pytest.mark.parametrize("n", [100, 1000])
def test_prefill_of_many_exponents(cuda_lib, n):
    """Exponents all over the format's range inside a key tile: one pass over the tile for each group of them."""
    s = Setup(4, 1, 16, 1, n, seed=n + 1)
    s.fill()
    s.model.exps[..., 0] = s.rng.integers(-30, -6, s.model.exps.shape[:-1])
    s.model.exps[..., 1] = s.rng.integers(-64, 8, s.model.exps.shape[:-1])
    s.upload()
    q = bf16(s.rng.standard_normal((50, 4, 128)))
    prefill_and_check(s, q, [50], [n])
    prefill_and_check(s, q, [50], [n], window=1)
    prefill_and_check(s, q, [50], [n], window=17, sinks=3)
    s.pool.close()


@pytest.mark.parametrize("n", [40, 1000])
def test_decode_of_many_exponents(cuda_lib, n):
    """One visible token, or a few, whose V exponents lie far apart: the lse keeps its precision."""
    s = Setup(4, 1, 16, 2, n, seed=n + 2)
    s.fill()
    s.model.exps[..., 0] = s.rng.integers(-30, -6, s.model.exps.shape[:-1])
    s.model.exps[..., 1] = s.rng.integers(-64, 8, s.model.exps.shape[:-1])
    s.upload()
    q = bf16(s.rng.standard_normal((2, 4, 128)))
    for m in range(n, n - 33, -1):
        decode_and_check(s, q, [m, m // 2], window=1)
        decode_and_check(s, q, [m, m // 2], window=17, sinks=3)
    s.pool.close()


@pytest.mark.parametrize("page", [16, 32])
def test_pages_given_up_behind_the_window(cuda_lib, page):
    """Pages that no query sees any more may be gone from the table: no error, the same output."""
    s = Setup(8, 2, page, 2, 2000, seed=page)
    s.fill()
    n, window, sinks = [2000, 1003], 300, 20
    q1, q2 = bf16(s.rng.standard_normal((2, 8, 128))), bf16(s.rng.standard_normal((110, 8, 128)))
    want1, want2 = s.decode(q1, n, window, sinks), s.prefill(q2, [60, 50], n, window, sinks)
    table = s.table.copy()
    for b, m in ((0, 60), (1, 50)):
        first = n[b] - m - window + 1                     # the first key that the earliest query's window shows
        table[b, -(-sinks // page):first // page] = -1
        table[b, -(-n[b] // page):] = s.pages + 7         # and pages that are not there yet
    got1, got2 = s.decode(q1, n, window, sinks, table=table), s.prefill(q2, [60, 50], n, window, sinks, table=table)
    for got, want in ((got1, want1), (got2, want2)):
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])
    assert s.pool.error() == 0
    s.pool.close()


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 300, 5), (900, 0), (899, 0),
                                          (50, 2 ** 31 - 1), (50, 800)])
def test_windows_and_first_tokens_beyond_the_sequence(cuda_lib, window, sinks):
    """Windows and counts of first tokens up to the largest integer, with queries before the first position too."""
    s = Setup(8, 2, 16, 2, 900, seed=12)
    s.fill()
    n = [900, 333]
    decode_and_check(s, bf16(s.rng.standard_normal((2, 8, 128))), n, window, sinks)
    count = [300, 340]                                    # the second sequence's first seven see nothing
    prefill_and_check(s, bf16(s.rng.standard_normal((640, 8, 128))), count, n, window, sinks, sample=150)
    s.pool.close()


def test_a_graph_with_copies_and_two_streams(cuda_lib):
    """Append, decode and prompt attention captured behind copies, one of them on another stream."""
    s = Setup(8, 2, 16, 1, 1100, seed=8, rope=dict(theta=1e4))
    s.fill()
    new_q, new_k = bf16(s.rng.standard_normal((40, 8, 128))), bf16(s.rng.standard_normal((40, 2, 128)))
    q, k, q_out = torch.zeros_like(new_q), torch.zeros_like(new_k), torch.zeros_like(new_q)
    out1, out2 = torch.zeros_like(new_q[:1]), torch.zeros_like(new_q)
    cu, start, n, table = i32([0, 40]), i32([1060]), i32([1100]), i32(s.table)
    pool, side, scale = s.pool.handle, torch.cuda.Stream(), 1 / math.sqrt(128)
    need = max(native.kv_decode_workspace_bytes(pool, 1, 1100), native.kv_prefill_workspace_bytes(pool, 1, 40, 1100))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        q.copy_(new_q)
        with torch.cuda.stream(side):
            k.copy_(new_k)
        here.wait_stream(side)
        native.kv_append_fp8(pool, 0, 1, q, 1024, k, 256, k, 256, cu, start, table, s.width, 40, q_out)
        native.kv_decode_attention_fp8(pool, 0, 1, q_out[39:], n, table, s.width, 1100, scale, 0, 0, out1, None, ws, need)
        native.kv_prefill_attention_fp8(pool, 0, 1, q_out, cu, n, table, s.width, 40, 1100, scale, 0, 0, out2, None, ws, need)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                         # before any eager call of these shapes
        step()
    for _ in range(5):
        for x in (q, k, q_out, out1, out2):
            x.zero_()
        graph.replay()
    torch.cuda.synchronize()
    got = out1.clone(), out2.clone()
    for x in (q, k, q_out, out1, out2):
        x.zero_()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out1) and torch.equal(got[1], out2) and out1.any() and s.pool.error() == 0
    s.model.codes[...], s.model.exps[...] = s.codes.cpu().numpy(), s.exps.cpu().numpy()
    s.check_rows(q_out[39:], [(0, 1099)], f64(out1), s.decode(q_out[39:], [1100])[1], 0, 0, lens=[1100])
    s.pool.close()


def test_attention_over_codes_beyond_32_bits(cuda_lib):
    """Pages past 2^32 bytes of codes attend as the same pages at the pool's start."""
    s = Setup(8, 8, 16, 2, 700, seed=3, spare=0)
    s.fill()
    q1, q2 = bf16(s.rng.standard_normal((2, 8, 128))), bf16(s.rng.standard_normal((150, 8, 128)))
    want1, want2 = s.decode(q1, [700, 333]), s.prefill(q2, [90, 60], [700, 333])
    pages = 140000                                        # 8 heads x 4096 B a page: 4.6 GB
    far = native.KVPool(native.KV_POOL_FP8, 1, 8, 8, 16, pages, 2)
    codes, exps = far.fp8_views(0)
    codes[pages - s.pages:].copy_(s.codes)
    exps[pages - s.pages:].copy_(s.exps)
    near, s.pool = s.pool, far
    table = s.table + (pages - s.pages)
    got1, got2 = s.decode(q1, [700, 333], table=table), s.prefill(q2, [90, 60], [700, 333], table=table)
    for got, want in ((got1, want1), (got2, want2)):
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])
    near.close()
    far.close()


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 12)])
def test_a_served_sequence(cuda_lib, window, sinks):
    """Prompt chunks and single tokens as a server runs them: append, attend, append, ..."""
    rope = dict(rotary_dim=128, theta=1e6)
    s = Setup(8, 2, 32, 2, 320, rope=rope, seed=7)
    at = np.array([0, 0])
    for count in ([200, 70], [1, 33], [1, 1], [60, 1], [1, 1], [1, 1]):
        T = sum(count)
        qkv = bf16(s.rng.standard_normal((T, 12, 128)))
        qo = s.append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], at, count)
        check_codes(s, fc.append(s.model, s.rope, f64(qkv[:, 8:10]), f64(qkv[:, 10:]), at, count, s.table))
        at = at + count
        if count == [1, 1]:
            decode_and_check(s, qo, at.tolist(), window, sinks)
        prefill_and_check(s, qo, count, at.tolist(), window, sinks, sample=60)
    assert s.pool.error() == 0
    s.pool.close()


def test_rotation_in_front_of_the_int2_path(cuda_lib):
    """kv_rope_apply in front of kv_append_bf16 and its decode: scores depend on distances alone, so a
    sequence moved by 1000 positions decodes to the same output."""
    rng = np.random.default_rng(0)
    pool = native.KVPool(native.KV_POOL_BF16, 1, 4, 2, 16, 8, 2)
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(rotary_dim=128, theta=1e4))
    n = 50
    k = bf16(np.tile(rng.standard_normal((n, 2, 128)), (2, 1, 1)))
    v = bf16(np.tile(rng.standard_normal((n, 2, 128)), (2, 1, 1)))
    pos = np.r_[0:n, 1000:1000 + n]
    kr = torch.empty_like(k)
    native.kv_rope_apply(pool.handle, 0, 2 * n, i32(pos), None, 0, k, 256, None, 0, kr, 256)
    pt = i32(np.arange(8).reshape(2, 4))
    native.kv_append_bf16(pool.handle, 0, 2, kr, v, i32([0, n, 2 * n]), i32([0, 0]), pt, 4, n)
    q = bf16(np.tile(rng.standard_normal((1, 4, 128)), (2, 1, 1)))
    native.kv_rope_apply(pool.handle, 0, 2, i32([n - 1, 1000 + n - 1]), q, 512, None, 0, q, 512, None, 0)
    wb = native.kv_decode_workspace_bytes(pool.handle, 2, n)
    ws = torch.empty(max(16, wb), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 4, 128, device="cuda")
    native.kv_decode_attention_bf16(pool.handle, 0, 2, q, i32([n, n]), pt, 4, n, 0.05, out, ws, wb)
    torch.cuda.synchronize()
    a, b = f64(out)
    # k and q rounded to bf16 after the rotation: 2^-8 of each product, scale 0.05 over 128 channels
    bound = 2 * 2 * 2.0 ** -8 * 0.05 * float(np.max(np.abs(f64(kr)).sum(-1))) * float(np.abs(f64(q)).max())
    assert np.abs(a - b).max() <= bound * np.abs(f64(v)).max()
    pool.close()
