// Single-token attention over the 8-bit cache.
#include "kv_fp8_simple.cuh"

namespace kvint2 {

namespace {

struct DecodeFp8Args {
  Fp8Layer L;
  AttnCall c;
  int B, Hq, G;
  int* err;
};

__global__ void __launch_bounds__(256) decode_fp8_kernel(DecodeFp8Args a) {
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= a.B * a.Hq) return;
  const int b = row / a.Hq, hq = row - b * a.Hq;
  int n = a.c.seq_len[b];
  if (n < 0 || n > a.c.max_len) {
    flag_error(a.err, KV_DEVERR_LENGTH);
    n = min(max(n, 0), a.c.max_len);
  }
  attend_row(a.L, a.c.pt + (size_t)b * a.c.max_pages, a.c.max_pages, hq / a.G,
             static_cast<const uint16_t*>(a.c.q) + (size_t)row * 128, n - 1, a.c.window, a.c.n_sink, a.c.scale,
             static_cast<uint16_t*>(a.c.out) + (size_t)row * 128, a.c.lse ? a.c.lse + row : nullptr, a.err, lane);
}

}  // namespace

size_t decode_fp8_workspace(const Pool& p, int B, int max_len) { return 16; }

cudaError_t launch_decode_fp8(const Pool& p, const Fp8Store& f, int layer, int B, const AttnCall& c, cudaStream_t s) {
  DecodeFp8Args a{fp8_layer(p, f, layer), c, B, p.cfg.num_q_heads, p.G, p.err};
  decode_fp8_kernel<<<(unsigned)(((long long)B * a.Hq + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvint2
