"""Refusals of the 8-bit cache's entry points that need a pool: nothing is launched."""

import ctypes

import pytest
import torch

from bit_kv_cache_12_gb300 import native as n

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rig(cuda_lib):
    pool = n.KVPool(n.KV_POOL_FP8, 2, 8, 2, 16, 8, 4)
    x = torch.zeros(64, 8, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    yield pool, x, i, ws
    torch.cuda.synchronize()
    pool.close()


def status(f, *a):
    try:
        f(*a)
    except n.KVError as e:
        return e.status
    return n.KV_OK


def changed(args, **kw):
    return [kw.get(k, v) for k, v in args.items()]


def test_rope_config(rig):
    pool = rig[0].handle

    def st(**kw):
        return status(n.kv_pool_set_rope, pool, 0, n.rope_config(**kw))
    assert st() == n.KV_OK
    for bad in (dict(rotary_dim=-32), dict(rotary_dim=160), dict(theta=1.0), dict(theta=float("nan")),
                dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=float("inf")),
                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_max_position=4096, beta_fast=1.0, beta_slow=2.0),
                dict(attention_factor=-1.0), dict(attention_factor=float("nan")), dict(rotary_dim=32, inv_freq=[float("inf")] * 16)):
        assert st(**bad) == n.KV_ERR_INVALID_ARG, bad
    assert st(rotary_dim=48) == n.KV_ERR_UNSUPPORTED
    c = n.rope_config()
    c.style = 2
    assert status(n.kv_pool_set_rope, pool, 0, c) == n.KV_ERR_INVALID_ARG
    c.style, c.scaling = 0, 4
    assert status(n.kv_pool_set_rope, pool, 0, c) == n.KV_ERR_INVALID_ARG
    assert status(n.kv_pool_set_rope, pool, 2, n.rope_config()) == n.KV_ERR_INVALID_ARG
    n.kv_pool_set_rope(pool, 0, n.rope_config(rotary_dim=0))


def test_rope_apply(rig):
    pool, x, i, _ = rig
    y = torch.empty_like(x)
    a = dict(pool=pool.handle, layer=0, n=4, pos=i, q=x, qs=1024, k=None, ks=0, qo=y, qos=1024, ko=None, kos=0)
    assert status(n.kv_rope_apply, *a.values()) == n.KV_OK
    assert status(n.kv_rope_apply, *changed(a, n=0, pos=None)) == n.KV_OK
    for bad in (dict(layer=2), dict(layer=-1), dict(n=-1), dict(pos=None), dict(q=None), dict(qo=None), dict(qs=1016),
                dict(qs=1028), dict(q=x.data_ptr() + 2), dict(qo=y.data_ptr() + 8), dict(k=x), dict(qo=x, qos=2048),
                dict(q=None, qo=None)):
        assert status(n.kv_rope_apply, *changed(a, **bad)) == n.KV_ERR_INVALID_ARG, bad


def test_append(rig):
    pool, x, i, _ = rig
    y = torch.empty_like(x)
    a = dict(pool=pool.handle, layer=0, n=1, q=x, qs=1024, k=x, ks=1024, v=x, vs=1024, cu=i, start=i, pt=i, w=4, most=0, qo=y)
    assert status(n.kv_append_fp8, *a.values()) == n.KV_OK
    assert status(n.kv_append_fp8, *changed(a, n=0, k=None, v=None, q=None, qo=None)) == n.KV_OK
    for bad in (dict(layer=2), dict(n=-1), dict(w=0), dict(most=-1), dict(k=None), dict(v=None), dict(cu=None), dict(start=None),
                dict(pt=None), dict(q=None), dict(qo=None), dict(ks=248), dict(vs=260), dict(qs=512), dict(k=x.data_ptr() + 4),
                dict(qo=y.data_ptr() + 2), dict(qo=x, qs=2048), dict(n=1 << 20, most=1 << 30)):
        assert status(n.kv_append_fp8, *changed(a, **bad)) == n.KV_ERR_INVALID_ARG, bad


def test_attention(rig):
    pool, x, i, ws = rig
    y = torch.empty_like(x)
    d = dict(pool=pool.handle, layer=0, B=4, q=x, n=i, pt=i, w=4, most=64, scale=0.1, window=0, sinks=0, out=y, lse=None, ws=ws,
             wb=ws.numel())
    assert status(n.kv_decode_attention_fp8, *d.values()) == n.KV_OK
    p = dict(pool=pool.handle, layer=0, B=4, q=x, cu=i, n=i, pt=i, w=4, mq=0, most=64, scale=0.1, window=0, sinks=0, out=y,
             lse=None, ws=ws, wb=ws.numel())
    assert status(n.kv_prefill_attention_fp8, *p.values()) == n.KV_OK
    for f, a in ((n.kv_decode_attention_fp8, d), (n.kv_prefill_attention_fp8, p)):
        for bad in (dict(layer=2), dict(B=0), dict(B=5), dict(q=None), dict(n=None), dict(pt=None), dict(w=0), dict(most=65),
                    dict(most=-1), dict(scale=float("nan")), dict(window=-1), dict(sinks=-1), dict(out=None), dict(ws=None),
                    dict(wb=0), dict(q=x.data_ptr() + 2), dict(out=y.data_ptr() + 8), dict(ws=ws.data_ptr() + 4),
                    dict(lse=ws.data_ptr() + 1)):
            assert status(f, *changed(a, **bad)) == n.KV_ERR_INVALID_ARG, (f.__name__, bad)
    assert status(n.kv_prefill_attention_fp8, *changed(p, cu=None)) == n.KV_ERR_INVALID_ARG
    assert status(n.kv_prefill_attention_fp8, *changed(p, mq=-1)) == n.KV_ERR_INVALID_ARG
    assert n.kv_decode_workspace_bytes(pool.handle, 5, 64) == 0
    assert n.kv_prefill_workspace_bytes(pool.handle, 5, 1, 64) == 0


def test_prompt_bounds_beyond_the_longest_sequence(rig):
    """A bound on the queries that no sequence can have is refused: the row numbers it stands for pass 32 bits."""
    pool, x, i, ws = rig
    y = torch.empty_like(x)
    for most_q in (6553601, 1 << 28, (1 << 31) - 1):
        assert status(n.kv_prefill_attention_fp8, pool.handle, 0, 4, x, i, i, i, 4, most_q, 64, 0.1, 0, 0, y, None, ws,
                      ws.numel()) == n.KV_ERR_INVALID_ARG
        assert n.kv_prefill_workspace_bytes(pool.handle, 1, most_q, 64) == 0
    assert n.kv_prefill_workspace_bytes(pool.handle, 1, 6553600, 64) > 0
    wide = n.KVPool(n.KV_POOL_FP8, 1, 64, 8, 16, 8, 4096)        # 6553600 queries of 4096 sequences: 2^32.6 blocks
    assert status(n.kv_prefill_attention_fp8, wide.handle, 0, 4096, x, i, i, i, 4, 6553600, 64, 0.1, 0, 0, y, None, ws,
                  ws.numel()) == n.KV_ERR_INVALID_ARG
    assert n.kv_prefill_workspace_bytes(wide.handle, 4096, 6553600, 64) == 0
    wide.close()


def test_other_kinds_of_pool(rig):
    _, x, i, ws = rig
    y = torch.empty_like(x)
    other = n.KVPool(n.KV_POOL_BF16, 1, 8, 2, 16, 8, 4)
    bad = n.KV_ERR_INVALID_ARG
    assert status(n.kv_append_fp8, other.handle, 0, 1, x, 1024, x, 1024, x, 1024, i, i, i, 4, 0, y) == bad
    assert status(n.kv_decode_attention_fp8, other.handle, 0, 1, x, i, i, 4, 64, 0.1, 0, 0, y, None, ws, ws.numel()) == bad
    assert status(n.kv_prefill_attention_fp8, other.handle, 0, 1, x, i, i, i, 4, 0, 64, 0.1, 0, 0, y, None, ws, ws.numel()) == bad
    assert status(n.kv_pool_get_fp8_layout, other.handle, 0) == bad
    assert n.kv_prefill_workspace_bytes(other.handle, 1, 1, 64) == 0
    # and the other kinds' calls refuse an FP8 pool
    fp8 = rig[0].handle
    assert status(n.kv_decode_attention_bf16, fp8, 0, 1, x, i, i, 4, 64, 0.1, y, ws, ws.numel()) == bad
    assert status(n.kv_append_bf16, fp8, 0, 1, x, x, i, i, i, 4, 0) == bad
    assert status(n.kv_append_quantize, fp8, 0, 1, x, x, i, i, i, 4, 0) == bad
    lay = n.kv_pool_get_layout(fp8, 0)
    assert not any(getattr(lay, f) for f in ("hist", "sink_k", "sink_v", "recent_k", "recent_v", "bf16_k", "bf16_v"))
    other.close()
