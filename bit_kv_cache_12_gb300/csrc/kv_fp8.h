// Internal declarations of the 8-bit cache: its storage beside the pool, the
// rotary parameters of a layer, and the launchers.
#pragma once

#include "kv_internal.h"

namespace kvint2 {

constexpr int kFp8TileBytes = 4096;   // e4m3 codes of one 16-token tile: K 2048 B, V 2048 B

// Storage of an FP8 pool: codes [layer][page][head][tile][K, V][2048], exponents
// [layer][page][head][tile][K, V].
struct Fp8Store {
  uint8_t* codes = nullptr;
  int8_t* exps = nullptr;
  size_t layer_stride = 0, exp_layer_stride = 0;   // bytes
};

// Rotary positions of a layer as the kernels take them (a kernel parameter).
struct RopeParams {
  unsigned long long turn[64];   // turns per position, modulo 1, in units of 2^-64
  float att = 1.f;               // factor on cos and sin
  float att2 = 1.f;              // its square
  int rd = 0;                    // rotated channels: 0, 32, 64, 96 or 128
  int interleaved = 0;
};

// One layer of an FP8 pool, as the attention kernels take it.
struct Fp8Layer {
  const uint8_t* codes;
  const int8_t* exps;
  long long num_pages;
  int Hkv, P;
};
inline Fp8Layer fp8_layer(const Pool& p, const Fp8Store& f, int layer) {
  return {f.codes + (size_t)layer * f.layer_stride, f.exps + (size_t)layer * f.exp_layer_stride, p.cfg.num_pages,
          p.cfg.num_kv_heads, p.cfg.page_size};
}

// Every kernel of the 8-bit cache is launched as the programmatic dependent of the
// one before it and lets the next one launch at once: a kernel's CTAs come up while
// the last ones of its predecessor finish.  Each of its threads passes
// after_predecessor() before it reads what the caller passes or writes anything,
// so a grid never ends before its predecessor.
// cluster: CTAs per cluster.
template <class... P>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster,
                             const P&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void release_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The layer's parameters from a configuration, or the reason it is refused.
kv_status_t rope_params(const kv_rope_config_t& c, RopeParams* out);

struct RopeRows {            // a [tokens][heads][128] bf16 operand and where its rotated rows go
  const void* in;
  int64_t in_stride;
  void* out;
  int64_t out_stride;
};
cudaError_t launch_rope(const Pool& p, const RopeParams& r, int n_tokens, const int32_t* positions, const RopeRows& q,
                        const RopeRows& k, cudaStream_t s);
cudaError_t launch_append_fp8(const Pool& p, const Fp8Store& f, const RopeParams& r, int layer, int n_seqs,
                              const RopeRows& q, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* cu, const int32_t* start, const int32_t* pt, int max_pages,
                              int max_tokens, cudaStream_t s);

// The arguments the two attention calls share.
struct AttnCall {
  const void* q;             // bf16 rows [rows][Hq][128]
  const int32_t* seq_len;
  const int32_t* pt;
  int max_pages, max_len;
  float scale;
  int window, n_sink;
  void* out;                 // bf16 rows
  float* lse;                // or NULL
  void* ws;
};
// A window that reaches from the last position back to the first hides nothing: none
// (and what is left keeps the kernels' positions minus windows in 32 bits).
inline int effective_window(int window, int max_len) { return window >= max_len ? 0 : window; }

// Whether a reference M (base 2) is so large that the roundings of logits and reference,
// each half a step of |M|, could carry a weight out of fp16's range: from there on weights
// come from the logit as it was rounded when it was compared with M, so that the largest
// one is in [2^0, 2^15] whatever the steps are.  Below, where a step is 2^-3 at most, they
// come from the product and ev - M in one rounding, which is closer.
__device__ __forceinline__ bool large_reference(float M) { return fabsf(M) > 0x1p20f && M > -2.9e38f; }

// ln(2^M l): M stands near -eV and log2 l near eV (up to 64), so l's exponent is
// added to M before its mantissa's logarithm (fp32 near 64 has steps of 2^-18).
__device__ __forceinline__ float lse_of(float M, float l) {
  if (l == 0.f) return -INFINITY;
  int e;
  const float m = frexpf(l, &e);
  return ((M + (float)e) + log2f(m)) * 0.6931471805599453f;
}

// What a call needs, and what every call up to these bounds does.
size_t decode_fp8_workspace(const Pool& p, int B, int max_len);
size_t decode_fp8_workspace_up_to(const Pool& p, int B, int max_len);
cudaError_t launch_decode_fp8(const Pool& p, const Fp8Store& f, int layer, int B, const AttnCall& c, cudaStream_t s);
size_t prefill_fp8_workspace(const Pool& p, int n_seqs, int max_q, int max_len);
size_t prefill_fp8_workspace_up_to(const Pool& p, int n_seqs, int max_q, int max_len);
cudaError_t launch_prefill_fp8(const Pool& p, const Fp8Store& f, int layer, int n_seqs, const int32_t* cu_q,
                               int max_q, const AttnCall& c, cudaStream_t s);

}  // namespace kvint2
