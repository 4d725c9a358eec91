"""Refusals of the 4-bit cache's entry points and of prompt attention that need a pool: nothing is launched."""

import pytest
import torch

from bit_kv_cache_12_gb300 import native as n
from tests.test_gpu_fp8_refusals import changed, status

pytestmark = pytest.mark.gpu
BAD = n.KV_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def rig(cuda_lib):
    pool = n.KVPool(n.KV_POOL_FP4, 2, 8, 2, 16, 8, 4)
    x = torch.zeros(64, 8, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    yield pool, x, i, ws
    torch.cuda.synchronize()
    pool.close()


def test_range_and_axes(rig):
    p = rig[0].handle
    assert status(n.kv_pool_set_fp4_range, p, 1, 32, -32) == n.KV_OK
    for a in ((2, 0, 0), (-1, 0, 0), (0, 33, 0), (0, 0, -33)):
        assert status(n.kv_pool_set_fp4_range, p, *a) == BAD
    assert status(n.kv_pool_set_rope_axes, p, 0, 1, [0] * 64) == BAD                 # no rotary positions yet
    n.kv_pool_set_rope(p, 0, n.rope_config(rotary_dim=64))
    assert status(n.kv_pool_set_rope_axes, p, 0, 3, [0, 1, 2, 2] * 8) == n.KV_OK
    for axes, axis in ((0, [0] * 32), (5, [0] * 32), (3, [0, 3] * 16), (3, [0, -1] * 16), (3, [0] * 31), (3, [0] * 33),
                       (3, [0] * 64), (3, [])):
        assert status(n.kv_pool_set_rope_axes, p, 0, axes, axis) == BAD, (axes, axis)
    assert status(n.kv_pool_set_rope_axes, p, 2, 1, [0] * 32) == BAD
    n.kv_pool_set_rope(p, 0, n.rope_config(rotary_dim=0))


def test_rope_apply_axes(rig):
    pool, x, i, _ = rig
    y = torch.empty_like(x)
    a = dict(pool=pool.handle, layer=0, n=4, pos=i, ps=4, q=x, qs=1024, k=None, ks=0, qo=y, qos=1024, ko=None, kos=0)
    assert status(n.kv_rope_apply_axes, *a.values()) == n.KV_OK
    assert status(n.kv_rope_apply_axes, *changed(a, n=0, pos=None)) == n.KV_OK
    for bad in (dict(layer=2), dict(layer=-1), dict(n=-1), dict(pos=None), dict(ps=3), dict(q=None), dict(qo=None), dict(qs=1016),
                dict(qs=1028), dict(q=x.data_ptr() + 2), dict(qo=y.data_ptr() + 8), dict(k=x), dict(qo=x, qos=2048),
                dict(q=None, qo=None)):
        assert status(n.kv_rope_apply_axes, *changed(a, **bad)) == BAD, bad


def test_append_and_read(rig):
    pool, x, i, _ = rig
    w = dict(pool=pool.handle, layer=0, n=1, k=x, ks=1024, v=x, vs=1024, cu=i, start=i, pt=i, w=4, most=0)
    r = dict(pool=pool.handle, layer=0, n=1, cu=i, start=i, pt=i, w=4, most=0, k=x, ks=1024, v=x, vs=1024)
    for f, a in ((n.kv_append_fp4, w), (n.kv_read_fp4, r)):
        assert status(f, *a.values()) == n.KV_OK
        assert status(f, *changed(a, n=0, k=None, v=None)) == n.KV_OK
        for bad in (dict(layer=2), dict(n=-1), dict(w=0), dict(most=-1), dict(cu=None), dict(start=None), dict(pt=None),
                    dict(k=None, v=None), dict(ks=248), dict(vs=260), dict(k=x.data_ptr() + 4), dict(v=x.data_ptr() + 8),
                    dict(n=1 << 20, most=1 << 30)):
            assert status(f, *changed(a, **bad)) == BAD, (f.__name__, bad)
    assert status(n.kv_append_fp4, *changed(w, k=None)) == BAD
    assert status(n.kv_append_fp4, *changed(w, v=None)) == BAD
    assert status(n.kv_read_fp4, *changed(r, v=None)) == n.KV_OK


def test_decode(rig):
    pool, x, i, ws = rig
    y = torch.empty_like(x)
    a = dict(pool=pool.handle, layer=0, B=4, q=x, n=i, pt=i, w=4, most=64, scale=0.1, window=0, sinks=0, out=y, lse=None, ws=ws,
             wb=ws.numel())
    assert status(n.kv_decode_attention_fp4, *a.values()) == n.KV_OK
    for bad in (dict(layer=2), dict(B=0), dict(B=5), dict(q=None), dict(n=None), dict(pt=None), dict(w=0), dict(most=65),
                dict(most=-1), dict(scale=float("nan")), dict(window=-1), dict(sinks=-1), dict(out=None), dict(ws=None),
                dict(wb=0), dict(q=x.data_ptr() + 2), dict(out=y.data_ptr() + 8), dict(ws=ws.data_ptr() + 4),
                dict(lse=ws.data_ptr() + 1)):
        assert status(n.kv_decode_attention_fp4, *changed(a, **bad)) == BAD, bad
    assert n.kv_decode_workspace_bytes(pool.handle, 5, 64) == 0


def test_prompt(rig):
    pool, x, i, ws = rig
    y = torch.empty_like(x)
    a = dict(pool=pool.handle, n=4, q=x, qs=1024, qr=64, k=x, ks=1024, v=x, vs=1024, kr=64, cq=i, ck=i, mq=64, mk=64, scale=0.1,
             window=0, sinks=0, out=y, lse=None, ws=ws, wb=ws.numel())
    assert status(n.kv_prompt_attention, *a.values()) == n.KV_OK
    assert status(n.kv_prompt_attention, *changed(a, mq=0)) == n.KV_OK
    for bad in (dict(n=0), dict(n=5), dict(q=None), dict(k=None), dict(v=None), dict(cq=None), dict(ck=None), dict(mq=-1),
                dict(mk=-1), dict(mq=6553601), dict(mk=6553601), dict(qs=1016), dict(ks=248), dict(vs=260), dict(qs=1 << 31),
                dict(ks=1 << 31), dict(vs=1 << 40), dict(qr=-1), dict(kr=0), dict(qr=1 << 31), dict(kr=1 << 31),
                dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(out=None), dict(ws=None), dict(wb=0),
                dict(q=x.data_ptr() + 2), dict(k=x.data_ptr() + 8), dict(v=x.data_ptr() + 4), dict(out=y.data_ptr() + 8),
                dict(ws=ws.data_ptr() + 4), dict(lse=ws.data_ptr() + 1)):
        assert status(n.kv_prompt_attention, *changed(a, **bad)) == BAD, bad
    assert n.kv_prompt_workspace_bytes(pool.handle, 5, 1, 64) == 0
    assert n.kv_prompt_workspace_bytes(pool.handle, 1, 6553601, 64) == 0
    assert n.kv_prompt_workspace_bytes(pool.handle, 1, 64, 6553601) == 0


def test_other_kinds_of_pool(rig):
    pool, x, i, ws = rig
    for kind in (0, 1, 2):
        other = n.KVPool(kind, 1, 8, 2, 16, 8, 4)
        h = other.handle
        assert status(n.kv_append_fp4, h, 0, 1, x, 1024, x, 1024, i, i, i, 4, 0) == BAD
        assert status(n.kv_read_fp4, h, 0, 1, i, i, i, 4, 0, x, 1024, x, 1024) == BAD
        assert status(n.kv_decode_attention_fp4, h, 0, 1, x, i, i, 4, 64, 0.1, 0, 0, x, None, ws, ws.numel()) == BAD
        assert status(n.kv_pool_get_fp4_layout, h, 0) == BAD
        assert status(n.kv_pool_set_fp4_range, h, 0, 0, 0) == BAD
        other.close()
    fp4 = pool.handle
    assert status(n.kv_append_fp8, fp4, 0, 1, x, 1024, x, 1024, x, 1024, i, i, i, 4, 0, x) == BAD
    assert status(n.kv_decode_attention_fp8, fp4, 0, 1, x, i, i, 4, 64, 0.1, 0, 0, x, None, ws, ws.numel()) == BAD
    assert status(n.kv_prefill_attention_fp8, fp4, 0, 1, x, i, i, i, 4, 0, 64, 0.1, 0, 0, x, None, ws, ws.numel()) == BAD
    assert status(n.kv_pool_get_fp8_layout, fp4, 0) == BAD
    assert status(n.kv_decode_attention_bf16, fp4, 0, 1, x, i, i, 4, 64, 0.1, x, ws, ws.numel()) == BAD
    assert status(n.kv_append_bf16, fp4, 0, 1, x, x, i, i, i, 4, 0) == BAD
    assert status(n.kv_append_quantize, fp4, 0, 1, x, x, i, i, i, 4, 0) == BAD
    lay = n.kv_pool_get_layout(fp4, 0)
    assert not any(getattr(lay, f) for f in ("hist", "sink_k", "sink_v", "recent_k", "recent_v", "bf16_k", "bf16_v"))
