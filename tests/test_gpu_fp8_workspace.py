"""One workspace, sized for the largest batch, serves every smaller call."""

import numpy as np
import pytest
import torch

from bit_kv_cache_12_gb300 import native
from tests.fp8_util import Setup, bf16, f64, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 8), (8, 8)])
def test_sizes_never_fall(cuda_lib, hq, hkv):
    pool = native.KVPool(native.KV_POOL_FP8, 1, hq, hkv, 16, 16, 600)
    lens = [0, 16, 256, 257, 1024, 2048, 2049, 4096, 32768, 131072, 6553600]
    decode = np.array([[native.kv_decode_workspace_bytes(pool.handle, b, n) for n in lens] for b in range(1, 601)])
    assert (decode > 0).all() and (np.diff(decode, axis=0) >= 0).all() and (np.diff(decode, axis=1) >= 0).all()
    queries = [0, 1, 7, 32, 33, 64, 65, 128, 257, 1000, 5000, 6553600]
    seqs = [1, 2, 3, 5, 8, 13, 19, 38, 39, 76, 77, 152, 600]
    prompt = np.array([[[native.kv_prefill_workspace_bytes(pool.handle, s, m, n) for n in lens] for m in queries] for s in seqs])
    assert (prompt > 0).all()
    for axis in range(3):
        assert (np.diff(prompt, axis=axis) >= 0).all()
    pool.close()


def test_a_workspace_for_the_largest_batch_serves_smaller_ones(cuda_lib):
    s = Setup(8, 8, 16, 3, 3000, seed=1)
    s.fill()
    big = native.KVPool(native.KV_POOL_FP8, 1, 8, 8, 16, s.pages, 300)
    for mine, theirs in zip(big.fp8_views(0), (s.codes, s.exps)):
        mine.copy_(theirs)
    need = native.kv_decode_workspace_bytes(big.handle, 300, 3000)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    q = bf16(s.rng.standard_normal((3, 8, 128)))
    for n in ([3000], [3000, 17], [3000, 1000, 2000]):
        out = torch.empty(len(n), 8, 128, dtype=torch.bfloat16, device="cuda")
        native.kv_decode_attention_fp8(big.handle, 0, len(n), q, i32(n), i32(s.table), s.width, 3000, 0.1, 0, 0, out, None, ws, need)
        np.testing.assert_array_equal(f64(out), s.decode(q, n, scale=0.1, max_len=3000)[0])
    need = native.kv_prefill_workspace_bytes(big.handle, 300, 4096, 3000)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    q = bf16(s.rng.standard_normal((90, 8, 128)))
    for count, n in (([3], [3000]), ([20, 4], [3000, 100]), ([60, 10, 20], [2000, 3000, 20])):
        out = torch.full((90, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        native.kv_prefill_attention_fp8(big.handle, 0, len(n), q, i32(np.r_[0, np.cumsum(count)]), i32(n), i32(s.table), s.width,
                                        max(count), 3000, 0.1, 0, 0, out, None, ws, need)
        np.testing.assert_array_equal(f64(out), s.prefill(q, count, n, scale=0.1, max_len=3000)[0])
    big.close()
    s.pool.close()
