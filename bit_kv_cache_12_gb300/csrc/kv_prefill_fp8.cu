// Prompt attention over the 8-bit cache.
#include "kv_fp8_simple.cuh"

namespace kvint2 {

namespace {

struct PrefillFp8Args {
  Fp8Layer L;
  AttnCall c;
  const int32_t* cu;
  int max_q, Hq, G;
  int* err;
};

__global__ void __launch_bounds__(256) prefill_fp8_kernel(PrefillFp8Args a) {
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const int c0 = a.cu[s], m = a.cu[s + 1] - c0;
  int n = a.c.seq_len[s];
  if (m < 0 || m > a.max_q) {
    flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return;
  }
  if (n < 0 || n > a.c.max_len) {
    flag_error(a.err, KV_DEVERR_LENGTH);
    n = min(max(n, 0), a.c.max_len);
  }
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int i = (int)(item / a.Hq), hq = (int)(item - (long long)i * a.Hq);
  if (i >= m) return;
  const size_t row = ((size_t)c0 + i) * a.Hq + hq;
  attend_row(a.L, a.c.pt + (size_t)s * a.c.max_pages, a.c.max_pages, hq / a.G,
             static_cast<const uint16_t*>(a.c.q) + row * 128, n - m + i, a.c.window, a.c.n_sink, a.c.scale,
             static_cast<uint16_t*>(a.c.out) + row * 128, a.c.lse ? a.c.lse + row : nullptr, a.err, lane);
}

}  // namespace

size_t prefill_fp8_workspace(const Pool& p, int n_seqs, int max_q, int max_len) { return 16; }

cudaError_t launch_prefill_fp8(const Pool& p, const Fp8Store& f, int layer, int n_seqs, const int32_t* cu_q,
                               int max_q, const AttnCall& c, cudaStream_t s) {
  if (max_q == 0) return cudaSuccess;
  PrefillFp8Args a{fp8_layer(p, f, layer), c, cu_q, max_q, p.cfg.num_q_heads, p.G, p.err};
  prefill_fp8_kernel<<<dim3((unsigned)(((long long)max_q * a.Hq + 7) / 8), n_seqs), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvint2
