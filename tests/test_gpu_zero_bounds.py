"""A bound of 0 on the tokens or queries of a sequence is a bound like any other: a sequence that has some is
flagged, and nothing is stored or written."""

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from tests import fp4_util, fp8_util
from tests.fp8_util import bf16
from tests.test_gpu_prompt import Prompt

pytestmark = pytest.mark.gpu

KV_DEVERR_SEQ_RANGE = 3


@pytest.mark.parametrize("count", [[3, 0], [0, 40], [0, 0]])
def test_appends_and_reads(cuda_lib, count):
    error = KV_DEVERR_SEQ_RANGE if any(count) else 0
    s = fp4_util.Setup(8, 2, 16, 2, 64, seed=1)
    s.fill()
    k, v = (bf16(s.rng.standard_normal((43, 2, 128))) for _ in range(2))
    s.append(k, v, [5, 0], count, most=0)
    assert s.pool.error() == error
    s.check_tiles()
    got = s.read([5, 0], count, most=0, rows=43)
    assert s.pool.error() == error and (got == 7).all()
    s.pool.close()
    s = fp8_util.Setup(8, 2, 16, 2, 64, seed=1)
    s.fill()
    q = bf16(s.rng.standard_normal((43, 8, 128)))
    q_out = s.append(q, k, v, [5, 0], count, most=0)
    assert s.pool.error() == error and (q_out == 7).all()
    np.testing.assert_array_equal(s.codes.cpu().numpy(), s.model.codes)
    s.pool.close()


@pytest.mark.parametrize("count", [[3, 0], [0, 40], [0, 0]])
def test_prompts(cuda_lib, count):
    error = KV_DEVERR_SEQ_RANGE if any(count) else 0
    p = Prompt(8, 2, count, [50, 60], seed=2, spare=3)
    out, lse = p.run(most=0)
    assert p.pool.error() == error and (out == 7).all() and (lse == 7).all()
    p.close()
    s = fp8_util.Setup(8, 2, 16, 2, 64, seed=3)
    s.fill()
    q = bf16(s.rng.standard_normal((43, 8, 128)))
    out, lse = torch.full_like(q, 7.0), torch.full((43, 8), 7.0, device="cuda")
    s.prefill(q, count, [50, 60], most=0, out=out, lse=lse)
    assert s.pool.error() == error and (out == 7).all() and (lse == 7).all()
    # (a length above its bound as well)
    s.prefill(q, [0, 0], [50, 60], most=0, max_len=55, out=out, lse=lse)
    assert s.pool.error() == 2 and (out == 7).all()
    s.pool.close()


def test_no_sequences(cuda_lib):
    for pool, append in ((native.KV_POOL_FP4, native.kv_append_fp4), (native.KV_POOL_FP8, native.kv_append_fp8)):
        x = native.KVPool(pool, 1, 8, 2, 16, 4, 2)
        q = () if pool == native.KV_POOL_FP4 else (None, 0)
        tail = () if pool == native.KV_POOL_FP4 else (None,)
        append(x.handle, 0, 0, *q, None, 256, None, 256, None, None, None, 4, 0, *tail)
        torch.cuda.synchronize()
        assert x.error() == 0
        x.close()
