"""A batch of chunks behind cached prefixes with one call of each operator: the chunks are appended, all of every
sequence is read back, and the chunks' own rows take the place of their stored ones before the attention."""

import math

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from oracle import fp8cache as fc
from tests.fp4_util import Setup
from tests.fp8_util import bf16, f64, i32
from tests.test_gpu_prompt import check_row

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,page,window,sinks", [(8, 2, 16, 0, 0), (16, 4, 32, 60, 8)])
def test_batch_of_chunks(cuda_lib, hq, hkv, page, window, sinks):
    prefix, count = [70, 0, 301, 33], [20, 45, 1, 130]
    end = [a + b for a, b in zip(prefix, count)]
    s = Setup(hq, hkv, page, 4, max(end), 1, -1, seed=page)
    s.fill()
    t = sum(count)
    q = bf16(s.rng.standard_normal((t, hq, 128)))
    k, v = (bf16(s.rng.standard_normal((t, hkv, 128))) for _ in range(2))
    before = [[s.model.rows(s.table[b], prefix[b], h) if prefix[b] else (np.zeros((0, 128)),) * 2 for h in range(hkv)]
              for b in range(4)]
    s.append(k, v, prefix, count)
    cu, ck = (np.concatenate([[0], np.cumsum(x)]) for x in (count, end))
    kv = s.read([0] * 4, end)
    own = np.concatenate([ck[b] + prefix[b] + np.arange(count[b]) for b in range(4)])
    at = torch.as_tensor(own).cuda()
    kv[0, at], kv[1, at] = k, v
    wb = native.kv_prompt_workspace_bytes(s.pool.handle, 4, max(count), max(end))
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(t, hq, device="cuda")
    native.kv_prompt_attention(s.pool.handle, 4, q, hq * 128, t, kv[0], hkv * 128, kv[1], hkv * 128, int(ck[-1]), i32(cu), i32(ck),
                               max(count), max(end), 1 / math.sqrt(128), window, sinks, out, lse, ws, wb)
    torch.cuda.synchronize()
    q, k, v, out, lse = (f64(x) for x in (q, k, v, out, lse))
    for b in range(4):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        for i in range(0, count[b], 9):
            see = fc.visible(prefix[b] + i, end[b], window, sinks)
            for h in range(hq):
                g = h // (hq // hkv)
                keys, values = (np.concatenate([before[b][g][w], x[rows, g]]) for w, x in enumerate((k, v)))
                check_row(out[cu[b] + i, h], lse[cu[b] + i, h], q[cu[b] + i, h], keys, values, see, 1 / math.sqrt(128), (b, i, h))
    assert s.pool.error() == 0
    s.pool.close()
