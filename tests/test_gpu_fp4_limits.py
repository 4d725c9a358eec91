"""The 4-bit cache's operators, prompt attention and rotary axes at their limits: caches and rows beyond 32-bit
offsets, the last positions, negative first rows, workspaces of the largest call, calls that overlap, graphs of
several calls, and views that outlive their pool's name."""

import gc
import itertools
import math
import weakref

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from tests.fp4_util import Setup
from tests.fp8_util import bf16, f64, i32
from tests.test_gpu_prompt import Prompt

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


def test_pages_beyond_32_bits(cuda_lib):
    """A cache of 4.8 GB whose sequences lie at its end: the bytes and rows of a small one."""
    s = Setup(16, 8, 32, 2, 300, seed=1)
    s.fill()
    count = 130000
    big = native.KVPool(native.KV_POOL_FP4, 1, 16, 8, 32, count, 2)
    view = big.fp4_view(0)
    assert view.numel() > 1 << 32
    shift = count - s.pages
    view[shift:].copy_(s.view)
    small, s.pool, s.view = (s.pool, s.view), big, view[shift:]
    table = s.table + shift
    k, v = (bf16(s.rng.standard_normal((160, 8, 128))) for _ in range(2))
    s.append(k, v, [30, 101], [100, 60], table=table)
    s.model.append(f64(k), f64(v), [30, 101], [100, 60], s.table)
    s.check_tiles()
    assert not view[:1000].any()
    got = f64(s.read([0, 0], [130, 161], table=table))
    for b, (at, n) in enumerate(((0, 130), (130, 161))):
        for h in range(8):
            for w in range(2):
                np.testing.assert_array_equal(got[w, at:at + n, h], s.model.rows(s.table[b], n, h)[w])
    q = bf16(s.rng.standard_normal((2, 16, 128)))
    out, lse = s.decode(q, [130, 161], table=table)
    s.check_rows(q, [(0, 129), (1, 160)], out, lse, 0, 0, lens=[130, 161])
    assert big.error() == 0
    big.close()
    small[0].close()


def test_rows_beyond_32_bits(cuda_lib):
    """Rows 2^27 elements apart: those of 20 tokens span 5.4 GB."""
    s = Setup(2, 2, 16, 1, 48, seed=2)
    native.kv_pool_set_rope(s.pool.handle, 0, native.rope_config(rotary_dim=128, theta=1e4))
    far = 1 << 27
    flat = torch.empty(20 * far, dtype=torch.bfloat16, device="cuda")
    a, b, c = (flat[256 * i:].as_strided((20, 2, 128), (far, 128, 1)) for i in range(3))
    for x in (a, b):
        x.copy_(bf16(s.rng.standard_normal((20, 2, 128))))
    s.append(a, b, [5], [20])
    s.model.append(f64(a), f64(b), [5], [20], s.table)
    s.check_tiles()
    near = s.read([5], [20])
    s.read([5], [20], out=(a, c))
    assert torch.equal(a, near[0]) and torch.equal(c, near[1])
    native.kv_rope_apply_axes(s.pool.handle, 0, 20, i32(np.arange(20)), 20, a, far, None, 0, c, far, None, 0)
    out = torch.empty(2, 20, 2, 128, dtype=torch.bfloat16, device="cuda")
    native.kv_rope_apply_axes(s.pool.handle, 0, 20, i32(np.arange(20)), 20, near[0], 256, None, 0, out[0], 256, None, 0)
    assert torch.equal(c, out[0])
    cu = i32([0, 20])
    wb = native.kv_prompt_workspace_bytes(s.pool.handle, 1, 20, 20)
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    for i, (q, k, v) in enumerate(((c, a, b), (c.contiguous(), a.contiguous(), b.contiguous()))):
        native.kv_prompt_attention(s.pool.handle, 1, q, q.stride(0), 20, k, k.stride(0), v, v.stride(0), 20, cu, cu, 20, 20,
                                   SCALE, 0, 0, out[i], None, ws, wb)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and s.pool.error() == 0
    s.pool.close()


def test_last_positions(cuda_lib):
    """Tokens up to position 2^31 - 2, and one more, which is refused on the device."""
    s = Setup(2, 1, 32, 1, 64, seed=3)
    s.fill()
    width = 1 << 26
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, -2:] = torch.as_tensor(s.table[0])
    base = (1 << 31) - 64
    k, v = (bf16(s.rng.standard_normal((40, 1, 128))) for _ in range(2))

    def call(start, n):
        native.kv_append_fp4(s.pool.handle, 0, 1, k, 128, v, 128, i32([0, n]), i32([start]), table, width, 40)
        out = torch.full((2, 40, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        native.kv_read_fp4(s.pool.handle, 0, 1, i32([0, n]), i32([start]), table, width, 40, out[0], 128, out[1], 128)
        torch.cuda.synchronize()
        return out

    got = call(base + 24, 39)                              # the last at 2^31 - 2
    s.model.append(f64(k[:39]), f64(v[:39]), [24], [39], s.table)
    s.check_tiles()
    assert s.pool.error() == 0
    want = s.model.rows(s.table[0], 63, 0)
    for w in range(2):
        np.testing.assert_array_equal(f64(got[w])[:39, 0], want[w][24:])
    assert (got[:, 39:] == 7).all()
    got = call(base + 24, 40)
    assert s.pool.error() == 3 and (got == 7).all()
    s.check_tiles()
    s.pool.close()


def test_negative_first_rows(cuda_lib):
    """Prefix sums below zero: those sequences are flagged and left out, the others are served."""
    s = Setup(4, 2, 16, 3, 48, seed=4)
    s.fill()
    k, v = (bf16(s.rng.standard_normal((20, 2, 128))) for _ in range(2))
    for cu in ([-9, -4, 0, 7], [-2 ** 31, 2 ** 31 - 1, 0, 7], [-1, 4, 0, 7], [2 ** 31 - 1, -2 ** 31, 0, 7]):
        s.append(k, v, [3, 3, 3], [5, 5, 7], cu=cu, most=7)
        assert s.pool.error() == 3
        s.model.append(f64(k[:7]), f64(v[:7]), [3], [7], s.table[2:])
        s.check_tiles()
        got = s.read([3, 3, 3], [5, 5, 7], cu=cu, most=7, rows=20)
        assert s.pool.error() == 3 and (got[:, 7:] == 7).all()
        for h in range(2):
            for w in range(2):
                np.testing.assert_array_equal(f64(got)[w, :7, h], s.model.rows(s.table[2], 10, h)[w][3:])
    s.pool.close()


@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 8), (8, 8)])
def test_workspace_sizes_never_fall(cuda_lib, hq, hkv):
    pool = native.KVPool(native.KV_POOL_FP4, 1, hq, hkv, 16, 16, 600)
    lens = [0, 1, 16, 256, 257, 1024, 2048, 2049, 4096, 32768, 131072, 6553600]
    decode = np.array([[native.kv_decode_workspace_bytes(pool.handle, b, n) for n in lens] for b in range(1, 601)])
    assert (decode > 0).all() and (np.diff(decode, axis=0) >= 0).all() and (np.diff(decode, axis=1) >= 0).all()
    queries = [0, 1, 7, 32, 33, 64, 65, 128, 257, 1000, 5000, 6553600]
    seqs = [1, 2, 3, 5, 8, 13, 19, 38, 39, 76, 77, 152, 600]
    prompt = np.array([[[native.kv_prompt_workspace_bytes(pool.handle, s, m, n) for n in lens] for m in queries] for s in seqs])
    assert (prompt > 0).all()
    for axis in range(3):
        assert (np.diff(prompt, axis=axis) >= 0).all()
    pool.close()


def test_one_workspace_serves_every_smaller_call(cuda_lib):
    """Batches, lengths and windows below the bounds; their results are those of a workspace of their own."""
    s = Setup(8, 2, 16, 60, 2500, seed=5)
    s.fill()
    need = native.kv_decode_workspace_bytes(s.pool.handle, 60, 2500)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    q = bf16(s.rng.standard_normal((60, 8, 128)))
    n = s.rng.integers(1, 2501, 60)
    for b, longest, window in itertools.product((1, 2, 7, 60), (2500, 600, 17), (0, 700, 33)):
        m = np.minimum(n[:b], longest)
        out = torch.empty(b, 8, 128, dtype=torch.bfloat16, device="cuda")
        native.kv_decode_attention_fp4(s.pool.handle, 0, b, q, i32(m), i32(s.table), s.width, longest, SCALE, window, 4, out,
                                       None, ws, need)
        np.testing.assert_array_equal(f64(out), s.decode(q[:b], m, window, 4, max_len=longest)[0])
    s.pool.close()


def test_calls_that_overlap(cuda_lib):
    """Decodes of two layers and two prompts on two streams at once, many times over: the bits of one at a time."""
    s = Setup(8, 2, 16, 4, 3000, layers=2, seed=6)
    s.fill()
    s.pool.fp4_view(1).copy_(s.view.flip(0))
    table, n = i32(s.table), i32([3000, 17, 1500, 2999])
    q = bf16(s.rng.standard_normal((4, 8, 128)))
    p = Prompt(8, 2, [100, 300], [2000, 300], seed=7)
    cq, ck = i32(p.cq), i32(p.ck)
    wd = native.kv_decode_workspace_bytes(s.pool.handle, 4, 3000)
    wp = native.kv_prompt_workspace_bytes(p.pool.handle, 2, 300, 2000)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(torch.empty(wd, dtype=torch.uint8, device="cuda"), torch.empty(wp, dtype=torch.uint8, device="cuda"),
             torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda"),
             torch.empty(400, 8, 128, dtype=torch.bfloat16, device="cuda")) for _ in range(2)]

    def calls(i, stream):
        d, w, out, rows = sets[i]
        native.kv_decode_attention_fp4(s.pool.handle, i, 4, q, n, table, s.width, 3000, SCALE, 0, 0, out, None, d, wd, stream)
        native.kv_prompt_attention(p.pool.handle, 2, p.q, p.q.stride(0), p.tq, p.k, p.k.stride(0), p.v, p.v.stride(0), p.tk, cq,
                                   ck, 300, 2000, SCALE, 0, 0, rows, None, w, wp, stream)

    want = []
    for i in range(2):
        calls(i, None)
        torch.cuda.synchronize()
        want.append([x.clone() for x in sets[i][2:]])
    assert not torch.equal(want[0][0], want[1][0]) and torch.equal(want[0][1], want[1][1])
    for _ in range(30):
        for i in range(2):
            calls(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(sets[i][2:], want[i]))
    assert s.pool.error() == 0
    p.close()
    s.pool.close()


def test_a_captured_step(cuda_lib):
    """Rotary axes, append and decode of a token in one graph, replayed with other rows, places and lengths."""
    s = Setup(8, 2, 16, 3, 200, seed=8)
    s.fill()
    native.kv_pool_set_rope(s.pool.handle, 0, native.rope_config(rotary_dim=64, theta=1e5))
    native.kv_pool_set_rope_axes(s.pool.handle, 0, 2, [i % 2 for i in range(32)])
    qkv = torch.empty(3, 12, 128, dtype=torch.bfloat16, device="cuda")
    rot = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    pos, start, n, cu, table = (i32(x) for x in (np.zeros((2, 3)), [0] * 3, [0] * 3, [0, 1, 2, 3], s.table))
    wb = native.kv_decode_workspace_bytes(s.pool.handle, 3, 200)
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 8, device="cuda")

    def step():
        native.kv_rope_apply_axes(s.pool.handle, 0, 3, pos, 3, qkv, 1536, qkv[:, 8:], 1536, rot, 1024, qkv[:, 8:], 1536)
        native.kv_append_fp4(s.pool.handle, 0, 3, qkv[:, 8:], 1536, qkv[:, 10:], 1536, cu, start, table, s.width, 1)
        native.kv_decode_attention_fp4(s.pool.handle, 0, 3, rot, n, table, s.width, 200, SCALE, 0, 0, out, lse, ws, wb)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    lens = np.array([0, 40, 199])
    for _ in range(2):
        x = bf16(s.rng.standard_normal((3, 12, 128)))
        qkv.copy_(x)
        pos.copy_(i32(s.rng.integers(0, 5000, (2, 3))))
        start.copy_(i32(lens))
        n.copy_(i32(lens + 1))
        g.replay()
        torch.cuda.synchronize()
        s.model.append(f64(qkv[:, 8:10]), f64(qkv[:, 10:]), lens, [1] * 3, s.table)
        s.check_tiles()
        s.check_rows(rot, [(b, m) for b, m in enumerate(lens)], f64(out), f64(lse), 0, 0, lens=lens + 1)
        lens = lens + [1, 1, -30]
    assert s.pool.error() == 0
    s.pool.close()


def test_axes_at_the_last_positions(cuda_lib):
    """Positions up to 2^31 - 1: the bits of kv_rope_apply at each axis' position."""
    pool = native.KVPool(native.KV_POOL_BF16, 1, 4, 1, 16, 1, 1)
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(rotary_dim=128, theta=1e6, style="interleaved"))
    axis = np.arange(64) % 2
    native.kv_pool_set_rope_axes(pool.handle, 0, 2, axis.tolist())
    rng = np.random.default_rng(9)
    x = bf16(rng.standard_normal((33, 4, 128)))
    pos = np.stack([2 ** 31 - 1 - np.arange(33), 2 ** 31 - 40 + np.arange(33)])
    one = [torch.empty_like(x) for _ in range(2)]
    for a in range(2):
        native.kv_rope_apply(pool.handle, 0, 33, i32(pos[a]), x, 512, None, 0, one[a], 512, None, 0)
    out = torch.empty_like(x)
    native.kv_rope_apply_axes(pool.handle, 0, 33, i32(pos), 33, x, 512, None, 0, out, 512, None, 0)
    torch.cuda.synchronize()
    first = torch.as_tensor(np.repeat(axis == 0, 2), device="cuda")
    assert torch.equal(out, torch.where(first, one[0], one[1]))
    pool.close()


def test_a_view_keeps_its_pool(cuda_lib):
    pool = native.KVPool(native.KV_POOL_FP4, 1, 2, 1, 16, 4, 1)
    ref, view = weakref.ref(pool), pool.fp4_view(0)
    del pool
    gc.collect()
    assert ref() is not None and not view.any()
    del view
    gc.collect()
    assert ref() is None
