"""Rotary positions and the append into the 8-bit cache, against the fp64 model."""

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc
from tests.fp8_util import Setup, bf16, check_codes, check_rotated, f64, i32

pytestmark = pytest.mark.gpu

YARN = dict(scaling="yarn", factor=4.0, original_max_position=32768)
ROPES = [dict(rotary_dim=128, style="half", theta=1e6), dict(rotary_dim=64, style="half", theta=1e4),
         dict(rotary_dim=96, style="half", theta=1e4, scaling="ntk", factor=8.0), dict(rotary_dim=32, style="half"),
         dict(rotary_dim=128, style="interleaved", theta=5e5, **YARN),
         dict(rotary_dim=64, style="interleaved", scaling="linear", factor=2.0), dict(rotary_dim=0),
         dict(rotary_dim=128, style="half", **YARN)]


@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("n", [1, 15, 16, 33, 200])
def test_rope_apply(cuda_lib, rope, n):
    s = Setup(hq=8, hkv=2, rope=rope)
    rng = np.random.default_rng(n)
    qkv = bf16(rng.standard_normal((n, 12, 128)))
    pos = rng.integers(0, [1, 1000, 131072, 2 ** 31 - 1][n % 4], n)
    pos[rng.random(n) < 0.2] = -1
    q, k = qkv[:, :8], qkv[:, 8:10]
    qo = torch.full((n, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")      # outputs with a stride of their own
    ko = torch.full((n, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    native.kv_rope_apply(s.pool.handle, 0, n, i32(pos), q, q.stride(0), k, k.stride(0), qo, qo.stride(0), ko, 256)
    torch.cuda.synchronize()
    live = pos >= 0
    for got, x in ((qo[:, :8], q), (ko, k)):
        assert (f64(got)[~live] == 7).all()
        check_rotated(f64(got)[live], f64(x)[live], s.rope, pos[live])
    assert (qo[:, 8:] == 7).all()
    # in place, and one operand alone
    want_q, want_k = qo[:, :8].clone(), ko.clone()
    want_q[~torch.as_tensor(live)] = q[~torch.as_tensor(live)]
    native.kv_rope_apply(s.pool.handle, 0, n, i32(pos), q, q.stride(0), None, 0, q, q.stride(0), None, 0)
    assert torch.equal(qkv[:, :8].view(torch.int16), want_q.view(torch.int16))
    k2 = torch.zeros_like(ko)
    native.kv_rope_apply(s.pool.handle, 0, n, i32(np.maximum(pos, 0)), None, 0, k, k.stride(0), None, 0, k2, 256)
    assert torch.equal(k2[torch.as_tensor(live)], want_k[torch.as_tensor(live)])
    s.pool.close()


def test_rope_of_other_pool_kinds_and_layers(cuda_lib):
    """Each layer has its own speeds; the pool's kind does not matter; custom speeds."""
    pool = native.KVPool(native.KV_POOL_INT2_3TIER, 2, 4, 2, 16, 4, 1)
    speeds = [0.5 / (i + 1) for i in range(16)]
    native.kv_pool_set_rope(pool.handle, 1, native.rope_config(rotary_dim=32, inv_freq=speeds, attention_factor=1.25))
    x = bf16(np.random.default_rng(0).standard_normal((5, 2, 128)))
    pos = np.array([0, 1, 2, 77, 123456])
    for layer, rope in ((0, fc.Rope(0)), (1, fc.Rope(32, inv_freq=speeds, attention_factor=1.25))):
        out = torch.empty_like(x)
        native.kv_rope_apply(pool.handle, layer, 5, i32(pos), None, 0, x, 256, None, 0, out, 256)
        check_rotated(f64(out), f64(x), rope, pos)
    pool.close()


@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("page", [16, 32])
def test_append_in_chunks(cuda_lib, rope, page):
    """Chunks of all kinds of lengths, growing scales, out of one fused projection."""
    s = Setup(hq=4, hkv=2, page=page, seqs=4, longest=200, rope=rope, seed=page)
    s.fill()
    rng, at = s.rng, np.array([0, 5, 16, 40])
    for count in ([1, 1, 1, 1], [16, 3, 0, 70], [40, 12, 33, 1], [0, 0, 17, 2]):
        T = sum(count)
        qkv = rng.standard_normal((T, 8, 128)) * np.exp(rng.standard_normal((T, 8, 1)))
        qkv = bf16(qkv)
        q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
        qo = s.append(q, k, v, at, count)
        check_codes(s, fc.append(s.model, s.rope, f64(k), f64(v), at, count, s.table))
        pos = np.concatenate([np.arange(a, a + c) for a, c in zip(at, count)])
        check_rotated(f64(qo), f64(q), s.rope, pos)
        at = at + count
    assert s.pool.error() == 0
    s.pool.close()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (8, 1), (40, 10), (64, 8)])
def test_append_head_counts(cuda_lib, hq, hkv):
    s = Setup(hq=hq, hkv=hkv, seqs=2, longest=64, rope=ROPES[0])
    k, v, q = (bf16(s.rng.standard_normal((37, h, 128))) for h in (hkv, hkv, hq))
    qo = s.append(q, k, v, [3, 0], [20, 17])
    check_codes(s, fc.append(s.model, s.rope, f64(k), f64(v), [3, 0], [20, 17], s.table))
    check_rotated(f64(qo), f64(q), s.rope, np.concatenate([np.arange(3, 23), np.arange(17)]))
    s.pool.close()


def test_append_without_q_in_place_and_padded(cuda_lib):
    s = Setup(hq=4, hkv=2, seqs=2, longest=64, rope=ROPES[0])
    q, k, v = (bf16(s.rng.standard_normal((40, h, 128))) for h in (4, 2, 2))
    s.append(None, k, v, [0, 0], [20, 11])
    check_codes(s, fc.append(s.model, s.rope, f64(k)[:31], f64(v)[:31], [0, 0], [20, 11], s.table))
    before = f64(q)
    s.append(q, k, v, [20, 11], [9, 0], q_out=q)          # rows from 9 on belong to nobody
    check_rotated(f64(q)[:9], before[:9], s.rope, np.arange(20, 29))
    np.testing.assert_array_equal(f64(q)[9:], before[9:])
    check_codes(s, fc.append(s.model, s.rope, f64(k)[:9], f64(v)[:9], [20, 11], [9, 0], s.table))
    s.pool.close()


def test_append_extremes(cuda_lib):
    """Zeros, tiny and huge values, NaN and infinity, exponents at both ends and at their borders."""
    s = Setup(hq=2, hkv=2, page=32, seqs=1, longest=160, rope=dict(rotary_dim=64, style="half"))
    k, v = s.rng.standard_normal((2, 150, 2, 128))
    k[0:16] = 0; v[0:16] = 0
    k[16:32] *= 1e-30; v[16:32] *= 2.0 ** -60
    k[40, 0] *= 1e6; v[41, 1] *= 1e30
    v[50, 0, 3] = np.nan; k[51, 1, 7] = np.inf; v[52, 1, 100] = -np.inf; k[53, 0, 127] = np.nan
    v[64:80] = 0; v[66, 0, 5] = 7.0; v[66, 1, 5] = 7.03125     # at the border of an exponent, and above it
    k[80:96] = np.nan                                          # a tile of nothing but NaN
    k, v = bf16(k), bf16(v)
    kk, vv = f64(k), f64(v)
    at = 0
    for c in (16, 25, 12, 1, 46, 50):
        s.append(None, k[at:at + c], v[at:at + c], [at], [c])
        check_codes(s, fc.append(s.model, s.rope, kk[at:at + c], vv[at:at + c], [at], [c], s.table))
        at += c
    assert s.exps.cpu().numpy()[s.table[0, 0], :, 0].tolist() == [[-64, -64], [-64, -64]]
    assert s.exps.cpu().numpy()[s.table[0, 2], :, 0, 1].tolist() == [-6, -5]
    assert s.pool.error() == 0
    s.pool.close()


def test_append_device_errors(cuda_lib):
    s = Setup(hq=2, hkv=2, page=16, seqs=3, longest=48, rope=ROPES[0])
    s.fill()
    q, k, v = (bf16(s.rng.standard_normal((40, 2, 128))) for _ in range(3))
    cases = [([0, 0, 40], [10, 12, 9], None, native, 3),               # the third leaves the table's span
             ([0, -1, 0], [10, 12, 9], None, None, 3), ([0, 2 ** 31 - 20, 0], [10, 12, 9], None, None, 3)]
    for start, count, _, _, code in cases:
        bad = 2 if start[2] else 1
        qo = s.append(q, k, v, start, count)
        keep = [c if i != bad else 0 for i, c in enumerate(count)]
        rows = np.concatenate([np.arange(10), np.arange(10, 22) if bad == 2 else np.arange(22, 31)])
        lost = np.setdiff1d(np.arange(31), rows)
        assert (f64(qo)[lost] == 7).all() and (f64(qo)[31:] == 7).all()
        check_codes(s, fc.append(s.model, s.rope, f64(k)[rows], f64(v)[rows], np.array(start) * (np.array(keep) > 0),
                                 keep, s.table))
        assert s.pool.error() == code
    table = s.table.copy()
    table[1, 0], table[0, 1] = s.pages, -1
    qo = s.append(q, k, v, [4, 0, 0], [20, 12, 8], table=table)
    check_codes(s, fc.append(s.model, s.rope, f64(k)[:40], f64(v)[:40], [4, 0, 0], [20, 12, 8], table))
    check_rotated(f64(qo), f64(q), s.rope, np.concatenate([np.arange(4, 24), np.arange(12), np.arange(8)]))
    assert s.pool.error() == 1
    # more tokens than the host said: the first ones are kept; a falling prefix sum is skipped
    s.append(q, k, v, [0, 0, 0], [5, 9, 3], most=5)
    rows = np.r_[0:5, 5:10, 14:17]
    check_codes(s, fc.append(s.model, s.rope, f64(k)[rows], f64(v)[rows], [0, 0, 0], [5, 5, 3], s.table))
    assert s.pool.error() == 3
    s.append(q, k, v, [0, 0, 0], [5, 9, 3], cu=[0, 5, 3, 6])
    rows = np.r_[0:5, 3:6]
    check_codes(s, fc.append(s.model, s.rope, f64(k)[rows], f64(v)[rows], [0, 0, 0], [5, 0, 3], s.table))
    assert s.pool.error() == 3
    s.pool.close()


def test_append_layers_streams_and_graph(cuda_lib):
    """Another layer of the pool, a side stream, and a captured append replayed on new tokens."""
    s = Setup(hq=4, hkv=2, seqs=2, longest=64, rope=ROPES[0], layers=3, layer=2)
    q, k, v = (bf16(s.rng.standard_normal((24, h, 128))) for h in (4, 2, 2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cu, start, table = i32([0, 14, 24]), i32([0, 7]), i32(s.table)
    qo = torch.empty(24, 4, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: native.kv_append_fp8(s.pool.handle, 2, 2, q, 512, k, 256, v, 256, cu, start, table,  # noqa: E731
                                        s.width, 14, qo)
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    check_codes(s, fc.append(s.model, s.rope, f64(k), f64(v), [0, 7], [14, 10], s.table))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    k.copy_(bf16(s.rng.standard_normal(k.shape) * 3))
    start.copy_(i32([14, 17]))
    g.replay()
    torch.cuda.synchronize()
    check_codes(s, fc.append(s.model, s.rope, f64(k), f64(v), [14, 17], [14, 10], s.table))
    check_rotated(f64(qo), f64(q), s.rope, np.r_[14:28, 17:27])
    for layer in (0, 1):
        c, e = s.pool.fp8_views(layer)
        assert not c.any() and not e.any()
    s.pool.close()


def test_code_offsets_beyond_32_bits(cuda_lib):
    """Pages past 2^32 bytes of codes."""
    pages = 140000                                             # 8 heads x 2 x 2048 B = 32 KB a page: 4.6 GB
    s = Setup(hq=8, hkv=8, page=16, seqs=1, longest=64, rope=ROPES[0], spare=0)
    pool = native.KVPool(native.KV_POOL_FP8, 1, 8, 8, 16, pages, 1)
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(**ROPES[0]))
    far = s.table + (pages - s.pages)
    k, v = (bf16(s.rng.standard_normal((50, 8, 128))) for _ in range(2))
    s.append(None, k, v, [0], [50], table=far, pool=pool)
    codes, exps = pool.fp8_views(0)
    s.codes, s.exps = codes[pages - s.pages:], exps[pages - s.pages:]
    check_codes(s, fc.append(s.model, s.rope, f64(k), f64(v), [0], [50], s.table))
    assert not codes[:1000].any()
    pool.close()
    s.pool.close()


def test_the_last_positions(cuda_lib):
    """Tokens up to position 2^31 - 2 are stored; a run that would pass it is refused, whatever the table spans."""
    near, far = (Setup(hq=4, hkv=1, page=16, seqs=1, longest=16, spare=0) for _ in range(2))
    k, v = (bf16(near.rng.standard_normal((8, 1, 128))) for _ in range(2))
    far.width = (1 << 27) + 1                                  # pages: 2^31 + 16 positions
    table = torch.zeros(1, far.width, dtype=torch.int32, device="cuda")
    cu, start = i32([0, 8]), i32([(1 << 31) - 8])
    call = lambda cu: native.kv_append_fp8(far.pool.handle, 0, 1, None, 0, k, 128, v, 128, cu, start, table, far.width, 8, None)
    call(cu)
    torch.cuda.synchronize()
    assert far.pool.error() == 3 and not far.codes.any()
    call(i32([0, 7]))
    near.append(None, k[:7], v[:7], [8], [7])
    assert far.pool.error() == 0 and near.pool.error() == 0
    assert near.codes.any() and torch.equal(near.codes, far.codes) and torch.equal(near.exps, far.exps)
    near.pool.close()
    far.pool.close()


def test_views_keep_their_pool(cuda_lib):
    """A view of the stored codes outlives the last name of its pool."""
    import gc
    import weakref
    pool = native.KVPool(native.KV_POOL_FP8, 1, 8, 8, 16, 64, 1)
    codes, exps = pool.fp8_views(0)
    codes.fill_(3)
    alive = weakref.ref(pool)
    f8 = codes.view(torch.float8_e4m3fn)
    del pool, codes, exps
    gc.collect()
    assert alive() is not None
    assert (f8.float() == 3 * 2.0 ** -9).all()
    del f8
    gc.collect()
    assert alive() is None
