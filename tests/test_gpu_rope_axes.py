"""Rotary positions with several axes, against the fp64 model."""

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp4cache as f4
from oracle import fp8cache as fc
from tests.fp8_util import bf16, check_rotated, f64, i32

pytestmark = pytest.mark.gpu

ROPES = [dict(rotary_dim=128, style="half", theta=1e6), dict(rotary_dim=64, style="half", theta=1e4),
         dict(rotary_dim=96, style="interleaved", theta=1e4, scaling="ntk", factor=8.0), dict(rotary_dim=32, style="interleaved"),
         dict(rotary_dim=128, style="interleaved", theta=5e5, scaling="yarn", factor=4.0, original_max_position=32768)]


class Axes(fc.Rope):
    """fc.Rope whose positions are [axes, n]."""

    def __init__(self, axis, **kw):
        super().__init__(**kw)
        self.axis = axis

    def rotate(self, x, pos):
        return f4.rotate_axes(self, self.axis, x, pos)


def axis_maps(n):
    return [(2, [i * 2 // n for i in range(n)]), (3, [i % 3 for i in range(n)]),
            (4, np.random.default_rng(n).integers(0, 4, n).tolist()), (1, [0] * n), (4, [2] * n)]


@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("n", [1, 15, 16, 33, 200])
def test_rope_apply_axes(cuda_lib, rope, n):
    pool = native.KVPool(native.KV_POOL_FP4, 2, 8, 2, 16, 1, 1)
    native.kv_pool_set_rope(pool.handle, 1, native.rope_config(**rope))
    rng = np.random.default_rng(n)
    for axes, axis in axis_maps(rope["rotary_dim"] // 2):
        native.kv_pool_set_rope_axes(pool.handle, 1, axes, axis)
        qkv = bf16(rng.standard_normal((n, 12, 128)))
        pos = rng.integers(0, [1, 1000, 131072, 2 ** 31 - 1][(n + axes) % 4], (axes, n))
        pos[rng.random((axes, n)) < 0.1] = -1
        live = (pos >= 0).all(0)
        wide = np.full((axes, n + 5), -7)                # rows of positions further apart than the tokens
        wide[:, :n] = pos
        q, k = qkv[:, :8], qkv[:, 8:10]
        qo = torch.full((n, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        ko = torch.full((n, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        native.kv_rope_apply_axes(pool.handle, 1, n, i32(wide), n + 5, q, q.stride(0), k, k.stride(0), qo, qo.stride(0), ko, 256)
        torch.cuda.synchronize()
        model = Axes(axis, **rope)
        for got, x in ((qo[:, :8], q), (ko, k)):
            assert (f64(got)[~live] == 7).all()
            check_rotated(f64(got)[live], f64(x)[live], model, pos[:, live])
        assert (qo[:, 8:] == 7).all()
        # in place, one operand alone
        want = torch.where(torch.as_tensor(live, device="cuda")[:, None, None], ko, k)
        native.kv_rope_apply_axes(pool.handle, 1, n, i32(pos), n, None, 0, k, k.stride(0), None, 0, k, k.stride(0))
        assert torch.equal(k.view(torch.int16), want.view(torch.int16))
    pool.close()


@pytest.mark.parametrize("kind", [0, 1, 2, 4])
def test_same_position_on_every_axis(cuda_lib, kind):
    """The bits of kv_rope_apply; setting the speeds anew takes the axes back to one; layers apart."""
    pool = native.KVPool(kind, 2, 8, 2, 16, 2, 1)
    cfg = native.rope_config(rotary_dim=128, theta=1e6)
    for layer in (0, 1):
        native.kv_pool_set_rope(pool.handle, layer, cfg)
    axis = [i % 3 for i in range(64)]
    native.kv_pool_set_rope_axes(pool.handle, 0, 3, axis)
    rng = np.random.default_rng(kind)
    x = bf16(rng.standard_normal((40, 8, 128)))
    pos = rng.integers(0, 100000, 40)
    out = [torch.empty_like(x) for _ in range(4)]
    native.kv_rope_apply(pool.handle, 0, 40, i32(pos), x, 1024, None, 0, out[0], 1024, None, 0)
    native.kv_rope_apply_axes(pool.handle, 0, 40, i32([pos] * 3), 40, x, 1024, None, 0, out[1], 1024, None, 0)
    native.kv_rope_apply_axes(pool.handle, 1, 40, i32(pos), 40, x, 1024, None, 0, out[2], 1024, None, 0)
    native.kv_pool_set_rope(pool.handle, 0, cfg)
    native.kv_rope_apply_axes(pool.handle, 0, 40, i32(pos), 40, x, 1024, None, 0, out[3], 1024, None, 0)
    for o in out[1:]:
        assert torch.equal(o.view(torch.int16), out[0].view(torch.int16))
    pool.close()


def test_axes_streams_and_graph(cuda_lib):
    pool = native.KVPool(native.KV_POOL_FP4, 1, 4, 2, 16, 1, 1)
    rope = dict(rotary_dim=128, theta=1e4)
    native.kv_pool_set_rope(pool.handle, 0, native.rope_config(**rope))
    axis = [i % 3 for i in range(64)]
    native.kv_pool_set_rope_axes(pool.handle, 0, 3, axis)
    rng = np.random.default_rng(1)
    q, pos = bf16(rng.standard_normal((50, 4, 128))), i32(rng.integers(0, 5000, (3, 50)))
    out = torch.empty_like(q)
    call = lambda s=None: native.kv_rope_apply_axes(pool.handle, 0, 50, pos, 50, q, 512, None, 0, out, 512, None, 0, s)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    check_rotated(f64(out), f64(q), Axes(axis, **rope), pos.cpu().numpy())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    pos.copy_(i32(rng.integers(0, 5000, (3, 50))))
    q.copy_(bf16(rng.standard_normal((50, 4, 128))))
    g.replay()
    torch.cuda.synchronize()
    check_rotated(f64(out), f64(q), Axes(axis, **rope), pos.cpu().numpy())
    pool.close()
