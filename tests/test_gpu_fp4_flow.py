"""The 4-bit cache's operators together, as a program serves with them: a prompt of text and image
tokens, a chunk behind it, single tokens, each step against the fp64 model of all of them."""

import math

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc
from tests.fp4_util import Setup
from tests.fp8_util import bf16, check_rotated, f64, i32
from tests.test_gpu_prompt import check_row as check_prompt_row
from tests.test_gpu_rope_axes import Axes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,page,window,sinks", [(8, 2, 16, 0, 0), (16, 2, 32, 60, 8)])
def test_prompt_chunk_tokens(cuda_lib, hq, hkv, page, window, sinks):
    s = Setup(hq, hkv, page, 2, 256, 0, -1, seed=page)
    rope = dict(rotary_dim=128, theta=1e6)
    axis = [i % 3 for i in range(64)]
    native.kv_pool_set_rope(s.pool.handle, 0, native.rope_config(**rope))
    native.kv_pool_set_rope_axes(s.pool.handle, 0, 3, axis)
    scale, g = 1 / math.sqrt(128), hq // hkv
    lens = [0, 0]
    for step, count in enumerate(([90, 33], [20, 100], [1, 1], [1, 1], [0, 17], [1, 1])):
        t = sum(count)
        qkv = bf16(s.rng.standard_normal((t, hq + 2 * hkv, 128)))
        pos = np.sort(s.rng.integers(0, 500, (3, t)), 1)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        row = qkv.stride(0)
        raw = f64(qkv)
        native.kv_rope_apply_axes(s.pool.handle, 0, t, i32(pos), t, q, row, k, row, q, row, k, row)
        torch.cuda.synchronize()
        check_rotated(f64(q), raw[:, :hq], Axes(axis, **rope), pos)
        check_rotated(f64(k), raw[:, hq:hq + hkv], Axes(axis, **rope), pos)
        cu = np.concatenate([[0], np.cumsum(count)])
        end = [a + b for a, b in zip(lens, count)]
        if max(count) > 1:
            # keys and values: the cached prefix read back, then the chunk's own rows
            ck = np.concatenate([[0], np.cumsum(end)])
            kv = torch.zeros(2, ck[-1], hkv, 128, dtype=torch.bfloat16, device="cuda")
            for b in range(2):
                if lens[b]:
                    part = kv[:, int(ck[b]):int(ck[b]) + lens[b]]
                    native.kv_read_fp4(s.pool.handle, 0, 1, i32([0, lens[b]]), i32([0]), i32(s.table[b]), s.width, lens[b],
                                       part[0], hkv * 128, part[1], hkv * 128)
                for w, x in enumerate((k, v)):
                    kv[w, int(ck[b]) + lens[b]:int(ck[b + 1])] = x[int(cu[b]):int(cu[b + 1])]
            wb = native.kv_prompt_workspace_bytes(s.pool.handle, 2, max(count), max(end))
            ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
            out = torch.empty(t, hq, 128, dtype=torch.bfloat16, device="cuda")
            lse = torch.empty(t, hq, device="cuda")
            native.kv_prompt_attention(s.pool.handle, 2, q, row, t, kv[0], hkv * 128, kv[1], hkv * 128, int(ck[-1]), i32(cu),
                                       i32(ck), max(count), max(end), scale, window, sinks, out, lse, ws, wb)
            torch.cuda.synchronize()
            fq, fo, fl = f64(q), f64(out), f64(lse)
            for b in range(2):
                for h in range(hkv):
                    cached = s.model.rows(s.table[b], lens[b], h) if lens[b] else (np.zeros((0, 128)),) * 2
                    keys, values = (np.concatenate([cached[w], f64(x)[int(cu[b]):int(cu[b + 1]), h]])
                                    for w, x in enumerate((k, v)))
                    for i in range(0, count[b], 7):
                        at = int(cu[b]) + i
                        see = fc.visible(lens[b] + i, end[b], window, sinks)
                        for u in range(g):
                            hh = h * g + u
                            check_prompt_row(fo[at, hh], fl[at, hh], fq[at, hh], keys, values, see, scale, (step, b, i, hh))
        s.append(k, v, lens, count)
        s.model.append(f64(k), f64(v), lens, count, s.table)
        s.check_tiles()
        lens = end
        if max(count) == 1:
            qq = q.contiguous()
            out, lse = s.decode(qq, lens, window, sinks)
            s.check_rows(qq, [(b, lens[b] - 1) for b in range(2)], out, lse, window, sinks, lens=lens)
    assert s.pool.error() == 0
    s.pool.close()
