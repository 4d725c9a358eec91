// Causal attention over packed bf16 rows: a warp per (query, head), key by key, with a
// running maximum and sum.
#include <algorithm>

#include "kv_device.cuh"
#include "kv_fp4.h"

namespace kvint2 {

namespace {

constexpr int kThreads = 256;

struct PromptArgs {
  PromptCall c;
  int Hq, Hkv;
  int* err;
};

__global__ void __launch_bounds__(kThreads) prompt_kernel(PromptArgs a) {
  release_successor();
  after_predecessor();
  const PromptCall& c = a.c;
  const long long per = ((long long)c.max_q * a.Hq + 7) / 8;
  const int s = (int)(blockIdx.x / per);
  const long long row = blockIdx.x % per * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, i = (int)(row / a.Hq), hq = (int)(row % a.Hq);
  const int q0 = c.cu_q[s], n = c.cu_q[s + 1] - q0, k0 = c.cu_k[s], m = c.cu_k[s + 1] - k0;
  if (n < 0 || n > c.max_q || m < 0 || m > c.max_k || q0 < 0 || (long long)q0 + n > c.q_rows || k0 < 0 ||
      (long long)k0 + m > c.kv_rows) {
    if (row == 0 && lane == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return;
  }
  if (i >= n) return;
  const int pos = m - n + i, h = hq / (a.Hq / a.Hkv);
  const uint2 qw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(c.q) + (q0 + i) * c.q_stride + hq * 128 + 4 * lane);
  const float f = c.scale * 1.4426950408889634f;
  const float q[4] = {bf16lo(qw.x) * f, bf16hi(qw.x) * f, bf16lo(qw.y) * f, bf16hi(qw.y) * f};
  float M = -3e38f, l = 0.f, o[4] = {};
  const int low = c.window ? max(pos - c.window + 1, 0) : 0;
  for (int j = 0; j <= pos; ++j) {
    if (j < low && j >= c.n_sink) j = low;
    const uint16_t* kp = static_cast<const uint16_t*>(c.k) + (k0 + j) * c.k_stride + h * 128 + 4 * lane;
    const uint16_t* vp = static_cast<const uint16_t*>(c.v) + (k0 + j) * c.v_stride + h * 128 + 4 * lane;
    const uint2 kw = *reinterpret_cast<const uint2*>(kp), vw = *reinterpret_cast<const uint2*>(vp);
    const float x = warp_sum_xor(q[0] * bf16lo(kw.x) + q[1] * bf16hi(kw.x) + q[2] * bf16lo(kw.y) + q[3] * bf16hi(kw.y), 1);
    const float top = fmaxf(M, x), old = exp2_neg(M - top), w = exp2_neg(x - top);
    M = top;
    l = l * old + w;
    o[0] = o[0] * old + w * bf16lo(vw.x);
    o[1] = o[1] * old + w * bf16hi(vw.x);
    o[2] = o[2] * old + w * bf16lo(vw.y);
    o[3] = o[3] * old + w * bf16hi(vw.y);
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  const __nv_bfloat162 y0 = __floats2bfloat162_rn(o[0] * r, o[1] * r), y1 = __floats2bfloat162_rn(o[2] * r, o[3] * r);
  const size_t at = (size_t)(q0 + i) * a.Hq + hq;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.out) + at * 128 + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
  if (c.lse && lane == 0) c.lse[at] = lse_of(M, l);
}

}  // namespace

size_t prompt_workspace(const Pool&, int, int, int) { return 16; }
size_t prompt_workspace_up_to(const Pool&, int, int, int) { return 16; }

cudaError_t launch_prompt(const Pool& p, const PromptCall& c, cudaStream_t s) {
  if (c.max_q == 0) return cudaSuccess;
  const long long blocks = ((long long)c.max_q * p.cfg.num_q_heads + 7) / 8 * c.n_seqs;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  PromptArgs a{c, p.cfg.num_q_heads, p.cfg.num_kv_heads, p.err};
  return launch_dependent(prompt_kernel, dim3((unsigned)blocks), kThreads, 0, s, 1, a);
}

}  // namespace kvint2
