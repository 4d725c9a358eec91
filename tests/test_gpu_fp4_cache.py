"""Writing tokens into the 4-bit cache and reading them back: the stored bytes equal the model's, bit by bit."""

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from tests.fp4_util import Setup
from tests.fp8_util import bf16, f64, i32

pytestmark = pytest.mark.gpu


def rows(s, t, size=1.0):
    """k, v as parts of one wider projection, channels of different sizes, every 16th row exact ties."""
    x = s.rng.standard_normal((t, 2 * s.hkv + 1, 128)) * size * np.exp(s.rng.standard_normal((t, 1, 1)))
    x[:, :, 64:80] *= 8
    tie = np.array([6.0, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 16) * size
    for m, i in enumerate(range(0, t, 16)):
        x[i] = tie * (1 + (m % 8) / 8)
    x = bf16(x)
    return x[:, :s.hkv], x[:, s.hkv + 1:]


def check_read(s, start, count):
    got = f64(s.read(start, count))
    row = 0
    for b, (p0, n) in enumerate(zip(start, count)):
        for h in range(s.hkv):
            want = s.model.rows(s.table[b], p0 + n, h)
            for w in range(2):
                np.testing.assert_array_equal(got[w, row:row + n, h], want[w][p0:])
        row += n


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (16, 8), (40, 10)])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("k_exp,v_exp", [(0, 0), (-4, 3)])
def test_append_and_read(cuda_lib, hq, hkv, page, k_exp, v_exp):
    """Ragged appends into a cache with stale bytes, continued at every kind of offset."""
    s = Setup(hq, hkv, page, 5, 150, k_exp, v_exp, seed=hkv + page)
    s.fill()
    lens = np.zeros(5, int)
    for count in ([1, 0, 17, 64, 130], [1, 1, 1, 1, 1], [30, 15, 16, 33, 2], [3, 100, 7, 5, 1], [1, 1, 1, 1, 1]):
        k, v = rows(s, sum(count), 2.0 ** k_exp)
        start = lens.tolist()
        s.append(k, v, start, count)
        s.model.append(f64(k), f64(v), start, count, s.table)
        s.check_tiles()
        check_read(s, start, count)
        lens += count
    check_read(s, [0] * 5, lens.tolist())
    check_read(s, [0, 3, 16, 31, 100], [0, 1, 20, 40, 30])
    assert s.pool.error() == 0
    s.pool.close()


def test_edges_of_the_format(cuda_lib):
    """Zeros, values under and beyond the range, the largest and smallest finite ones, NaN and infinities."""
    for e in (0, -32, 32, 5):
        s = Setup(2, 2, 16, 1, 48, e, e, seed=3)
        x = np.zeros((40, 2, 128))
        unit = 2.0 ** e
        x[0], x[1], x[2] = 2.0 ** -11 * unit, 6 * 2.0 ** -10 * unit, 6.1 * 2.0 ** -10 * unit
        x[3], x[4], x[5] = 3.38e38, -3.38e38, 1e-38
        x[6, :, ::2], x[6, :, 1::2] = 2688 * unit, -2700 * unit
        x[7] = 2688 * unit * s.rng.uniform(-1.2, 1.2, (2, 128))
        x[8, 0, 3], x[8, 1, 100] = np.nan, np.inf
        x[9, :, ::16] = -np.inf
        x[10] = np.array([1e-40, 3e-39] * 64)
        x[11] = s.rng.standard_normal((2, 128)) * 2.0 ** -7 * unit
        x[12:] = s.rng.standard_normal((28, 2, 128)) * 2.0 ** s.rng.integers(-12, 12, (28, 2, 1)) * unit
        k = bf16(x)
        s.append(k, k.clone(), [3], [40])
        s.model.append(f64(k), f64(k), [3], [40], s.table)
        s.check_tiles()
        got = f64(s.read([3], [40]))
        want = [s.model.rows(s.table[0], 43, h) for h in range(2)]
        for w in range(2):
            for h in range(2):
                y = f64(torch.as_tensor(want[h][w][3:]).to(torch.bfloat16))
                np.testing.assert_array_equal(got[w, :, h], y)
        s.pool.close()


def test_rows_and_pages_that_are_left_alone(cuda_lib):
    """Rows behind the last sequence, sequences out of range, bad pages."""
    s = Setup(8, 2, 16, 4, 64, seed=1)
    s.fill()
    k, v = rows(s, 40)
    # the second leaves the table's span, the third starts below 0
    s.append(k, v, [5, 60, -1, 0], [7, 9, 4, 10], cu=[0, 7, 16, 20, 30])
    assert s.pool.error() == 3
    s.model.append(f64(k[:7]), f64(v[:7]), [5], [7], s.table)
    s.model.append(f64(k[20:30]), f64(v[20:30]), [0], [10], s.table[3:])
    s.check_tiles()
    got = s.read([5, 60, -1, 0], [7, 9, 4, 10], cu=[0, 7, 16, 20, 30], rows=40)
    assert s.pool.error() == 3
    g = f64(got)
    for h in range(2):
        for w in range(2):
            np.testing.assert_array_equal(g[w, :7, h], s.model.rows(s.table[0], 12, h)[w][5:])
            np.testing.assert_array_equal(g[w, 20:30, h], s.model.rows(s.table[3], 10, h)[w])
    assert (got[:, 7:20] == 7).all() and (got[:, 30:] == 7).all()
    # longer than the bound: truncated
    s.append(k, v, [0], [40], most=20)
    assert s.pool.error() == 3
    s.model.append(f64(k[:20]), f64(v[:20]), [0], [20], s.table)
    s.check_tiles()
    got = s.read([0], [40], most=20)
    assert s.pool.error() == 3 and (got[:, 20:] == 7).all() and (got[:, :20] != 7).any()
    # a falling prefix sum
    s.append(k, v, [0, 0], [5, 5], cu=[5, 0, 5], most=5)
    assert s.pool.error() == 3
    s.model.append(f64(k[:5]), f64(v[:5]), [0], [5], s.table[1:])
    s.check_tiles()
    # bad pages
    table = s.table.copy()
    table[0, 1], table[1, 0] = -1, s.pages
    s.append(k, v, [0, 0], [20, 20], table=table)
    assert s.pool.error() == 1
    s.model.append(f64(k), f64(v), [0, 0], [20, 20], table)
    s.check_tiles()
    got = s.read([0, 0], [20, 20], table=table)
    assert s.pool.error() == 1 and (got[:, 16:36] == 7).all() and (got[:, :16] != 7).any() and (got[:, 36:] != 7).any()
    s.pool.close()


def test_one_output_empty_calls_and_strides(cuda_lib):
    s = Setup(4, 2, 16, 2, 40, seed=2)
    s.fill()
    cu, start, table = i32([0, 20, 50]), i32([0, 3]), i32(s.table)
    wide = torch.full((50, 5, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    call = lambda n, most, k, v: native.kv_read_fp4(  # noqa: E731
        s.pool.handle, 0, n, cu, start, table, s.width, most, k, 640, v, 640)
    call(2, 30, wide[:, 1:], None)
    both = s.read([0, 3], [20, 30])
    assert torch.equal(wide[:, 1:3], both[0]) and (wide[:, 0] == 7).all() and (wide[:, 3:] == 7).all()
    call(2, 30, None, wide[:, 3:])
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 3:], both[1])
    call(0, 30, wide, wide)
    call(2, 0, wide, wide)
    native.kv_append_fp4(s.pool.handle, 0, 0, None, 0, None, 0, None, None, None, 1, 5)
    torch.cuda.synchronize()
    s.check_tiles()
    s.pool.close()


def test_layers_streams_and_graph(cuda_lib):
    """Layers apart, another stream, and a graph of append and read replayed with other rows and places."""
    s = Setup(4, 2, 32, 2, 64, 1, -1, layers=3, layer=1, seed=4)
    s.fill()
    others = [s.pool.fp4_view(i).clone() for i in (0, 2)]
    side = torch.cuda.Stream()
    k, v = rows(s, 30)
    side.wait_stream(torch.cuda.current_stream())
    s.append(k, v, [0, 5], [10, 20], stream=side)
    s.model.append(f64(k), f64(v), [0, 5], [10, 20], s.table)
    s.check_tiles()
    k, v = k.contiguous().clone(), v.contiguous().clone()
    cu, start, table = i32([0, 10, 30]), i32([0, 5]), i32(s.table)
    out = torch.zeros(2, 30, 2, 128, dtype=torch.bfloat16, device="cuda")

    def call():
        native.kv_append_fp4(s.pool.handle, 1, 2, k, 256, v, 256, cu, start, table, s.width, 20)
        native.kv_read_fp4(s.pool.handle, 1, 2, cu, start, table, s.width, 20, out[0], 256, out[1], 256)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for at in ([7, 9], [30, 40], [0, 0]):
        k.copy_(bf16(s.rng.standard_normal((30, 2, 128))))
        v.copy_(bf16(s.rng.standard_normal((30, 2, 128))))
        start.copy_(i32(at))
        g.replay()
        torch.cuda.synchronize()
        s.model.append(f64(k), f64(v), at, [10, 20], s.table)
        s.check_tiles()
        for w in range(2):
            want = np.stack([np.concatenate([s.model.rows(s.table[b], at[b] + n, h)[w][at[b]:] for b, n in ((0, 10), (1, 20))])
                             for h in range(2)], 1)
            np.testing.assert_array_equal(f64(out[w]), want)
    for i, x in zip((0, 2), others):
        assert torch.equal(s.pool.fp4_view(i), x)
    s.pool.close()
