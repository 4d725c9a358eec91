// Internal declarations of the 4-bit cache and of attention over bf16 rows: storage
// beside the pool, rotary axes, and the launchers.
#pragma once

#include "kv_fp8.h"

namespace kvint2 {

// A stored tile: 16 tokens of one KV head; see include/kvint2.h.
constexpr int kFp4TileBytes = 2304;
constexpr int kFp4V = 1024, kFp4KScale = 2048, kFp4VScale = 2176;
constexpr int kFp4ExpMax = 32;        // of a layer's exponents, either side

// Storage of an FP4 pool: tiles [layer][page][head][tile of the page][2304].
struct Fp4Store {
  uint8_t* tiles = nullptr;
  size_t layer_stride = 0;            // bytes
};
// A layer's exponents of K and V (host).
struct Fp4Range {
  int k = 0, v = 0;
};

// One layer of an FP4 pool, as the kernels take it.
struct Fp4Layer {
  uint8_t* tiles;
  long long num_pages;
  int Hkv, P;
  int k_exp, v_exp;
};
inline Fp4Layer fp4_layer(const Pool& p, const Fp4Store& f, const Fp4Range& r, int layer) {
  return {f.tiles + (size_t)layer * f.layer_stride, p.cfg.num_pages, p.cfg.num_kv_heads, p.cfg.page_size, r.k, r.v};
}

// Which axis turns each rotated pair of a layer (a kernel parameter).
struct RopeAxes {
  int n = 1;
  alignas(4) uint8_t axis[64] = {};
};
cudaError_t launch_rope_axes(const Pool& p, const RopeParams& r, const RopeAxes& x, int n_tokens,
                             const int32_t* positions, int64_t pos_stride, const RopeRows& q, const RopeRows& k,
                             cudaStream_t s);

// The ragged tokens that an append writes or a read returns.
struct Fp4Tokens {
  int n_seqs;
  const int32_t *cu, *start, *pt;
  int max_pages, max_tokens;
};
struct Fp4Rows {                      // k and v rows, strides in elements
  void *k, *v;
  int64_t k_stride, v_stride;
};
cudaError_t launch_append_fp4(const Pool& p, const Fp4Layer& L, const Fp4Tokens& t, const Fp4Rows& in, cudaStream_t s);
cudaError_t launch_read_fp4(const Pool& p, const Fp4Layer& L, const Fp4Tokens& t, const Fp4Rows& out, cudaStream_t s);

// Splits of each (sequence, KV head), the workspace they need, and what any call up to these
// bounds needs.
int decode_fp4_splits(const Pool& p, int B, int max_len, int window, int n_sink);
size_t decode_fp4_workspace(const Pool& p, int B, int n_split);
size_t decode_fp4_workspace_up_to(const Pool& p, int B, int max_len);
cudaError_t launch_decode_fp4(const Pool& p, const Fp4Layer& L, int layer, int B, int n_split, const AttnCall& c,
                              cudaStream_t s);

// Attention of packed rows.
struct PromptCall {
  const void *q, *k, *v;              // bf16 rows
  int64_t q_stride, k_stride, v_stride;
  long long q_rows, kv_rows;
  const int32_t *cu_q, *cu_k;
  int n_seqs, max_q, max_k;
  float scale;
  int window, n_sink;
  void* out;
  float* lse;                         // or NULL
  void* ws;
};
size_t prompt_workspace(const Pool& p, int n_seqs, int max_q, int max_k);
size_t prompt_workspace_up_to(const Pool& p, int n_seqs, int max_q, int max_k);
cudaError_t launch_prompt(const Pool& p, const PromptCall& c, cudaStream_t s);

}  // namespace kvint2
