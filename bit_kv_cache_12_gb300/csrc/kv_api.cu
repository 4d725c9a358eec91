// C ABI of libkvint2: argument checks, pool storage, launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "kv_fp4.h"
#include "kv_internal.h"

using kvint2::Pool;

struct kv_pool {
  Pool p;
  kvint2::Fp8Store fp8;
  kvint2::Fp4Store fp4;
  kvint2::RopeParams* rope = nullptr;   // host, one per layer, as the two below
  kvint2::RopeAxes* axes = nullptr;
  kvint2::Fp4Range* range = nullptr;
};

namespace {

bool is_pow2_in(int v, int lo, int hi) { return v >= lo && v <= hi && (v & (v - 1)) == 0; }

kv_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? KV_OK : KV_ERR_CUDA; }

template <class T>
bool dev_alloc(T** ptr, size_t bytes) {
  if (bytes == 0) {
    *ptr = nullptr;
    return true;
  }
  void* v = nullptr;
  if (cudaMalloc(&v, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  *ptr = static_cast<T*>(v);
  return true;
}

void free_pool(kv_pool* pool) {
  Pool& p = pool->p;
  void* ptrs[] = {p.hist, p.sink_k, p.sink_v, p.rec_k,   p.rec_v,        p.bk,  p.bv,  p.Rk,
                  p.RvT,  p.clip,   p.rfrag,  p.tickets, p.step_tickets, p.arrive, p.err,
                  pool->fp8.codes, pool->fp8.exps, pool->fp4.tiles};
  for (void* q : ptrs)
    if (q) cudaFree(q);
  delete[] pool->rope;
  delete[] pool->axes;
  delete[] pool->range;
  delete pool;
}

__global__ void init_rotation_kernel(float* Rk, float* RvT, float* clip, size_t n_mat, size_t n_clip) {
  const size_t idx = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx < n_mat) {
    const int i = (int)((idx >> 7) & 127), c = (int)(idx & 127);
    const float v = (i == c) ? 1.f : 0.f;
    Rk[idx] = v;
    RvT[idx] = v;
  }
  if (idx < n_clip) clip[idx] = INFINITY;
}

bool valid_layer(const kv_pool_t* pool, int layer) {
  return pool && layer >= 0 && layer < pool->p.cfg.num_layers;
}

// KV_OK when the pool's device is the current one
kv_status_t on_pool_device(const Pool& p) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return KV_ERR_CUDA;
  return cur == p.device ? KV_OK : KV_ERR_INVALID_ARG;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// a [tokens][heads][128] bf16 operand: 16-byte rows, tokens `stride` elements apart
bool valid_rows(const void* p, int64_t stride, int heads) {
  return aligned16(p) && stride >= (int64_t)heads * 128 && (stride & 7) == 0;
}

// sequences and queries of a prompt call; its grid: a CTA per 256 rows and KV head
bool valid_prefill(const Pool& p, int32_t n_seqs, int32_t max_q) {
  if (n_seqs <= 0 || n_seqs > p.cfg.max_seqs || max_q < 0 || max_q > kvint2::kMaxDecodeLen) return false;
  return std::max<int64_t>(((int64_t)max_q * p.G + 255) / 256, 1) * n_seqs * p.cfg.num_kv_heads <= INT32_MAX;
}

// the arguments the two rotary calls share
kv_status_t check_rope(const kv_pool_t* pool, int layer, int n_tokens, const int32_t* positions,
                       const kvint2::RopeRows& q, const kvint2::RopeRows& k) {
  if (!valid_layer(pool, layer) || n_tokens < 0) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if ((q.in == nullptr) != (q.out == nullptr) || (k.in == nullptr) != (k.out == nullptr)) return KV_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!positions || (!q.in && !k.in))) return KV_ERR_INVALID_ARG;
  const int Hq = p.cfg.num_q_heads, Hkv = p.cfg.num_kv_heads;
  if (q.in && (!valid_rows(q.in, q.in_stride, Hq) || !valid_rows(q.out, q.out_stride, Hq))) return KV_ERR_INVALID_ARG;
  if (k.in && (!valid_rows(k.in, k.in_stride, Hkv) || !valid_rows(k.out, k.out_stride, Hkv))) return KV_ERR_INVALID_ARG;
  if ((q.in && q.in == q.out && q.in_stride != q.out_stride) || (k.in && k.in == k.out && k.in_stride != k.out_stride))
    return KV_ERR_INVALID_ARG;
  return on_pool_device(p);
}

// the arguments the 8-bit and the 4-bit decode share
kv_status_t check_decode(const kv_pool_t* pool, int kind, int layer, int B, const void* q, const int32_t* seq_len,
                         const int32_t* pt, int max_pages, int max_len, float scale, int window, int n_sink,
                         const void* out, const float* lse, const void* ws) {
  if (!valid_layer(pool, layer) || B <= 0 || max_pages <= 0 || max_len < 0) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != kind || B > p.cfg.max_seqs) return KV_ERR_INVALID_ARG;
  if (!q || !seq_len || !pt || !out || !ws) return KV_ERR_INVALID_ARG;
  if (window < 0 || n_sink < 0 || !std::isfinite(scale)) return KV_ERR_INVALID_ARG;
  if ((int64_t)max_len > (int64_t)max_pages * p.cfg.page_size || max_len > kvint2::kMaxDecodeLen)
    return KV_ERR_INVALID_ARG;
  if (!aligned16(ws) || !aligned16(q) || !aligned16(out) || ((uintptr_t)lse & 3)) return KV_ERR_INVALID_ARG;
  return KV_OK;
}

// the ragged tokens of a 4-bit append or read
kv_status_t check_fp4_tokens(const kv_pool_t* pool, int layer, int n_seqs, const int32_t* cu, const int32_t* start,
                             const int32_t* pt, int max_pages, int max_tokens) {
  if (!valid_layer(pool, layer) || n_seqs < 0 || max_pages <= 0 || max_tokens < 0) return KV_ERR_INVALID_ARG;
  if (pool->p.cfg.kind != KV_POOL_FP4) return KV_ERR_INVALID_ARG;
  if (n_seqs > 0 && (!cu || !start || !pt)) return KV_ERR_INVALID_ARG;
  if ((int64_t)n_seqs * (((int64_t)max_tokens + 30) / kvint2::kTile) > INT32_MAX) return KV_ERR_INVALID_ARG;
  return KV_OK;
}

// queries and keys of a prompt call; its grid: a CTA per 256 rows and KV head
bool valid_prompt(const Pool& p, int32_t n_seqs, int32_t max_q, int32_t max_k) {
  return valid_prefill(p, n_seqs, max_q) && max_k >= 0 && max_k <= kvint2::kMaxDecodeLen;
}

}  // namespace

extern "C" {

kv_status_t kv_pool_create(const kv_pool_config_t* cfg, void* stream, kv_pool_t** out) {
  if (!cfg || !out) return KV_ERR_INVALID_ARG;
  *out = nullptr;
  const kv_pool_config_t c = *cfg;
  if (c.kind != KV_POOL_INT2_3TIER && c.kind != KV_POOL_BF16 && c.kind != KV_POOL_FP8 && c.kind != KV_POOL_FP4)
    return KV_ERR_INVALID_ARG;
  if (c.num_layers <= 0 || c.num_kv_heads <= 0 || c.num_q_heads <= 0 || c.max_seqs <= 0 ||
      c.num_pages <= 0 || c.num_pages > (int64_t)INT32_MAX)
    return KV_ERR_INVALID_ARG;
  if (c.num_q_heads % c.num_kv_heads != 0) return KV_ERR_INVALID_ARG;
  if (c.head_dim != 128) return KV_ERR_UNSUPPORTED;
  if (c.page_size != 16 && c.page_size != 32) return KV_ERR_UNSUPPORTED;
  const int G = c.num_q_heads / c.num_kv_heads;
  if (!is_pow2_in(G, 1, 8)) return KV_ERR_UNSUPPORTED;
  if (c.kind == KV_POOL_INT2_3TIER) {
    if (c.group_size != 64 && c.group_size != 128) return KV_ERR_UNSUPPORTED;
    if (c.sink_tokens < 0 || c.recent_tokens <= 0 || c.sink_tokens > 4096 || c.recent_tokens > 4096)
      return KV_ERR_INVALID_ARG;
  }
  // more than any device holds; up to here no size below passes 64 bits
  const double heads = (double)c.num_layers * c.num_kv_heads;
  if (heads * c.num_pages * c.page_size > 0x1p45 || heads * c.max_seqs > 0x1p40) return KV_ERR_OOM;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KV_ERR_CUDA;
  kv_pool_t* pool = new (std::nothrow) kv_pool_t();
  if (!pool) return KV_ERR_OOM;
  Pool& p = pool->p;
  p.cfg = c;
  p.device = dev;
  p.G = G;
  cudaDeviceGetAttribute(&p.sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (p.sm_count <= 0) p.sm_count = 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t L = c.num_layers, H = c.num_kv_heads;
  bool ok = true;
  if (c.kind == KV_POOL_INT2_3TIER) {
    p.tile_bytes = 1024 + kvint2::kTile * 8 * (128 / c.group_size);
    p.page_bytes = H * (c.page_size / kvint2::kTile) * p.tile_bytes;
    p.hist_layer_stride = (size_t)c.num_pages * p.page_bytes;
    p.sink_layer_stride = (size_t)c.max_seqs * H * c.sink_tokens * 128;
    p.rec_layer_stride = (size_t)c.max_seqs * H * c.recent_tokens * 128;
    ok = ok && dev_alloc(&p.hist, L * p.hist_layer_stride);
    ok = ok && dev_alloc(&p.sink_k, L * p.sink_layer_stride * 2);
    ok = ok && dev_alloc(&p.sink_v, L * p.sink_layer_stride * 2);
    ok = ok && dev_alloc(&p.rec_k, L * p.rec_layer_stride * 2);
    ok = ok && dev_alloc(&p.rec_v, L * p.rec_layer_stride * 2);
    ok = ok && dev_alloc(&p.Rk, L * H * 128 * 128 * sizeof(float));
    ok = ok && dev_alloc(&p.RvT, L * H * 128 * 128 * sizeof(float));
    ok = ok && dev_alloc(&p.clip, L * 2 * H * 128 * sizeof(float));
    ok = ok && dev_alloc(&p.rfrag, L * H * kvint2::kFragBlocks * kvint2::rfrag_per_head() * sizeof(uint4));
  } else if (c.kind == KV_POOL_FP8) {
    const size_t tiles = (size_t)c.num_pages * H * (c.page_size / kvint2::kTile);
    pool->fp8.layer_stride = tiles * kvint2::kFp8TileBytes;
    pool->fp8.exp_layer_stride = tiles * 2;
    ok = ok && dev_alloc(&pool->fp8.codes, L * pool->fp8.layer_stride);
    ok = ok && dev_alloc(&pool->fp8.exps, L * pool->fp8.exp_layer_stride);
  } else if (c.kind == KV_POOL_FP4) {
    pool->fp4.layer_stride = (size_t)c.num_pages * H * (c.page_size / kvint2::kTile) * kvint2::kFp4TileBytes;
    ok = ok && dev_alloc(&pool->fp4.tiles, L * pool->fp4.layer_stride);
  } else {
    p.bf16_layer_stride = (size_t)c.num_pages * H * c.page_size * 128;
    ok = ok && dev_alloc(&p.bk, L * p.bf16_layer_stride * 2);
    ok = ok && dev_alloc(&p.bv, L * p.bf16_layer_stride * 2);
  }
  ok = ok && dev_alloc(&p.tickets, L * c.max_seqs * H * sizeof(unsigned));
  ok = ok && dev_alloc(&p.arrive, L * c.max_seqs * H * kvint2::kMaskWords * sizeof(unsigned));
  ok = ok && dev_alloc(&p.step_tickets, L * ((c.max_seqs + 127) / 128) * sizeof(unsigned));
  ok = ok && dev_alloc(&p.err, sizeof(int));
  if (ok) {                                    // (last: of more layers than the device holds the host may not hold these)
    pool->rope = new (std::nothrow) kvint2::RopeParams[L]();
    pool->axes = new (std::nothrow) kvint2::RopeAxes[L]();
    pool->range = new (std::nothrow) kvint2::Fp4Range[L]();
    ok = pool->rope && pool->axes && pool->range;
  }
  if (!ok) {
    free_pool(pool);
    return KV_ERR_OOM;
  }
  cudaError_t e = cudaSuccess;
  auto zero = [&](void* ptr, size_t bytes) {
    if (ptr && bytes && e == cudaSuccess) e = cudaMemsetAsync(ptr, 0, bytes, s);
  };
  zero(p.hist, L * p.hist_layer_stride);
  zero(p.sink_k, L * p.sink_layer_stride * 2);
  zero(p.sink_v, L * p.sink_layer_stride * 2);
  zero(p.rec_k, L * p.rec_layer_stride * 2);
  zero(p.rec_v, L * p.rec_layer_stride * 2);
  zero(p.bk, L * p.bf16_layer_stride * 2);
  zero(p.bv, L * p.bf16_layer_stride * 2);
  zero(pool->fp8.codes, L * pool->fp8.layer_stride);
  zero(pool->fp8.exps, L * pool->fp8.exp_layer_stride);
  zero(pool->fp4.tiles, L * pool->fp4.layer_stride);
  zero(p.tickets, L * c.max_seqs * H * sizeof(unsigned));
  zero(p.arrive, L * c.max_seqs * H * kvint2::kMaskWords * sizeof(unsigned));
  zero(p.step_tickets, L * ((c.max_seqs + 127) / 128) * sizeof(unsigned));
  zero(p.err, sizeof(int));
  if (e == cudaSuccess && c.kind == KV_POOL_INT2_3TIER) {
    const size_t n_mat = L * H * 128 * 128, n_clip = L * 2 * H * 128;
    init_rotation_kernel<<<(unsigned)((n_mat + 255) / 256), 256, 0, s>>>(p.Rk, p.RvT, p.clip, n_mat, n_clip);
    e = cudaGetLastError();
    for (int l = 0; l < c.num_layers && e == cudaSuccess; ++l) {
      const size_t off = (size_t)l * H * 128 * 128;
      e = kvint2::launch_rotation_prep(p, l, p.Rk + off, p.RvT + off, s);
    }
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    free_pool(pool);
    return KV_ERR_CUDA;
  }
  *out = pool;
  return KV_OK;
}

kv_status_t kv_pool_destroy(kv_pool_t* pool) {
  if (!pool) return KV_ERR_INVALID_ARG;
  cudaError_t e = cudaDeviceSynchronize();
  free_pool(pool);
  return cuda_status(e);
}

kv_status_t kv_pool_set_rotation(kv_pool_t* pool, int32_t layer, const float* R_k,
                                 const float* R_v, const float* clip_k, const float* clip_v,
                                 void* stream) {
  if (!valid_layer(pool, layer) || !R_k || !R_v || !clip_k || !clip_v) return KV_ERR_INVALID_ARG;
  Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_INT2_3TIER) return KV_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t H = p.cfg.num_kv_heads;
  float* cl = p.clip + (size_t)layer * 2 * H * 128;
  cudaError_t e = cudaMemcpyAsync(cl, clip_k, H * 128 * sizeof(float), cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(cl + H * 128, clip_v, H * 128 * sizeof(float), cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess) e = kvint2::launch_rotation_prep(p, layer, R_k, R_v, s);
  // decodes read the rotation before they wait for the kernel ahead of them:
  // the set-up is complete before this call returns
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return cuda_status(e);
}

kv_status_t kv_pool_get_layout(const kv_pool_t* pool, int32_t layer, kv_pool_layout_t* out) {
  if (!valid_layer(pool, layer) || !out) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  *out = kv_pool_layout_t{};
  if (p.cfg.kind == KV_POOL_INT2_3TIER) {
    out->hist = p.hist + (size_t)layer * p.hist_layer_stride;
    out->hist_layer_stride = p.hist_layer_stride;
    out->hist_page_stride = p.page_bytes;
    out->hist_head_stride = p.page_bytes / p.cfg.num_kv_heads;
    out->tile_bytes = p.tile_bytes;
    out->sink_k = p.sink_k + (size_t)layer * p.sink_layer_stride;
    out->sink_v = p.sink_v + (size_t)layer * p.sink_layer_stride;
    out->recent_k = p.rec_k + (size_t)layer * p.rec_layer_stride;
    out->recent_v = p.rec_v + (size_t)layer * p.rec_layer_stride;
    out->tier_layer_stride = p.sink_layer_stride * 2;
    out->recent_layer_stride = p.rec_layer_stride * 2;
  } else if (p.cfg.kind == KV_POOL_BF16) {
    out->bf16_k = p.bk + (size_t)layer * p.bf16_layer_stride;
    out->bf16_v = p.bv + (size_t)layer * p.bf16_layer_stride;
    out->bf16_layer_stride = p.bf16_layer_stride * 2;
  }
  return KV_OK;
}

kv_status_t kv_pool_get_error(kv_pool_t* pool, int32_t* device_error_code) {
  if (!pool || !device_error_code) return KV_ERR_INVALID_ARG;
  int v = 0;
  cudaError_t e = cudaMemcpy(&v, pool->p.err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(pool->p.err, 0, sizeof(int));
  if (e != cudaSuccess) return KV_ERR_CUDA;
  *device_error_code = v;
  return v ? KV_ERR_DEVICE : KV_OK;
}

kv_status_t kv_store_tier(kv_pool_t* pool, int32_t layer, int32_t tier, int32_t n_rows,
                          const void* k, const void* v, const int32_t* seq, const int32_t* slot,
                          void* stream) {
  if (!valid_layer(pool, layer) || (tier != 0 && tier != 1) || n_rows < 0) return KV_ERR_INVALID_ARG;
  if (pool->p.cfg.kind != KV_POOL_INT2_3TIER) return KV_ERR_INVALID_ARG;
  if (n_rows > 0 && (!k || !v || !seq || !slot)) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_store_tier(pool->p, layer, tier, n_rows, k, v, seq, slot,
                                               static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_quantize_pack_f32(kv_pool_t* pool, int32_t layer, int32_t tensor, int64_t n_rows,
                                 const float* x_rot, uint8_t* codes, void* scale_zero,
                                 void* stream) {
  if (!valid_layer(pool, layer) || (tensor != 0 && tensor != 1) || n_rows < 0)
    return KV_ERR_INVALID_ARG;
  if (pool->p.cfg.kind != KV_POOL_INT2_3TIER) return KV_ERR_INVALID_ARG;
  if (n_rows > 0 && (!x_rot || !codes || !scale_zero)) return KV_ERR_INVALID_ARG;
  if (((uintptr_t)x_rot & 15) || ((uintptr_t)scale_zero & 3)) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_quantize_pack(pool->p, layer, tensor, n_rows, x_rot, codes,
                                                  scale_zero, static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_append_quantize(kv_pool_t* pool, int32_t layer, int32_t n_seqs, const void* k,
                               const void* v, const int32_t* cu_tokens, const int32_t* hist_start,
                               const int32_t* page_table, int32_t max_pages_per_seq,
                               int32_t max_tokens_per_seq, void* stream) {
  if (!valid_layer(pool, layer) || n_seqs < 0 || max_pages_per_seq <= 0 || max_tokens_per_seq < 0)
    return KV_ERR_INVALID_ARG;
  if (pool->p.cfg.kind != KV_POOL_INT2_3TIER) return KV_ERR_INVALID_ARG;
  if (n_seqs > 0 && (!k || !v || !cu_tokens || !hist_start || !page_table)) return KV_ERR_INVALID_ARG;
  if (((uintptr_t)k & 15) || ((uintptr_t)v & 15)) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_append(pool->p, layer, n_seqs, k, v, cu_tokens, hist_start,
                                           page_table, max_pages_per_seq, max_tokens_per_seq,
                                           static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_append_step(kv_pool_t* pool, int32_t layer, int32_t B, const void* k_new,
                           const void* v_new, int32_t* sink_len, int32_t* hist_len,
                           int32_t* recent_len, int32_t* recent_start, const int32_t* page_table,
                           int32_t max_pages_per_seq, void* stream) {
  if (!valid_layer(pool, layer) || B < 0 || max_pages_per_seq <= 0) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_INT2_3TIER || B > p.cfg.max_seqs) return KV_ERR_INVALID_ARG;
  if (B > 0 && (!k_new || !v_new || !sink_len || !hist_len || !recent_len || !recent_start ||
                !page_table))
    return KV_ERR_INVALID_ARG;
  if (((uintptr_t)k_new & 7) || ((uintptr_t)v_new & 7)) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_append_step(p, layer, B, k_new, v_new, sink_len, hist_len,
                                                recent_len, recent_start, page_table,
                                                max_pages_per_seq,
                                                static_cast<cudaStream_t>(stream)));
}

size_t kv_decode_workspace_bytes(const kv_pool_t* pool, int32_t B, int32_t max_len) {
  if (!pool || B <= 0 || max_len < 0 || max_len > kvint2::kMaxDecodeLen || B > pool->p.cfg.max_seqs) return 0;
  const Pool& p = pool->p;
  if (p.cfg.kind == KV_POOL_FP8) return kvint2::decode_fp8_workspace_up_to(p, B, max_len);
  if (p.cfg.kind == KV_POOL_FP4) return kvint2::decode_fp4_workspace_up_to(p, B, max_len);
  kvint2::DecodePlan pl = p.cfg.kind == KV_POOL_INT2_3TIER ? kvint2::plan_decode_int2(p, B, max_len)
                                                           : kvint2::plan_decode_bf16(p, B, max_len);
  return pl.bytes;
}

kv_status_t kv_decode_attention(kv_pool_t* pool, int32_t layer, int32_t B, const void* q,
                                const int32_t* sink_len, const int32_t* hist_len,
                                const int32_t* recent_len, const int32_t* recent_start,
                                const int32_t* page_table, int32_t max_pages_per_seq,
                                int32_t max_hist_len, float softmax_scale, float* out,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_layer(pool, layer) || B <= 0 || max_pages_per_seq <= 0 || max_hist_len < 0)
    return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_INT2_3TIER || B > p.cfg.max_seqs) return KV_ERR_INVALID_ARG;
  if (!q || !sink_len || !hist_len || !recent_len || !recent_start || !page_table || !out ||
      !workspace)
    return KV_ERR_INVALID_ARG;
  if ((int64_t)max_hist_len > (int64_t)max_pages_per_seq * p.cfg.page_size || max_hist_len > kvint2::kMaxDecodeLen)
    return KV_ERR_INVALID_ARG;
  if (((uintptr_t)workspace & 15) || ((uintptr_t)q & 1)) return KV_ERR_INVALID_ARG;
  kvint2::DecodePlan pl = kvint2::plan_decode_int2(p, B, max_hist_len);
  if (workspace_bytes < pl.bytes) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_decode_int2(p, layer, B, q, sink_len, hist_len, recent_len,
                                                recent_start, page_table, max_pages_per_seq, pl,
                                                softmax_scale, out, workspace,
                                                static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_decode_attention_noalloc(kv_pool_t* pool, int32_t layer, int32_t B, const void* q,
                                        const int32_t* sink_len, const int32_t* hist_len,
                                        const int32_t* recent_len, const int32_t* recent_start,
                                        const int32_t* page_table, int32_t max_pages_per_seq,
                                        int32_t max_hist_len, float softmax_scale, float* out,
                                        void* stream) {
  if (!valid_layer(pool, layer) || B <= 0 || max_pages_per_seq <= 0 || max_hist_len < 0)
    return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_INT2_3TIER || B > p.cfg.max_seqs) return KV_ERR_INVALID_ARG;
  if (!q || !sink_len || !hist_len || !recent_len || !recent_start || !page_table || !out)
    return KV_ERR_INVALID_ARG;
  if ((int64_t)max_hist_len > (int64_t)max_pages_per_seq * p.cfg.page_size || max_hist_len > kvint2::kMaxDecodeLen)
    return KV_ERR_INVALID_ARG;
  if ((uintptr_t)q & 1) return KV_ERR_INVALID_ARG;
  // the scratch buffer looked up below is the current device's: it must be the pool's
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return KV_ERR_CUDA;
  if (cur != p.device) return KV_ERR_INVALID_ARG;
  kvint2::DecodePlan pl = kvint2::plan_decode_int2(p, B, max_hist_len);
  void* scratch = nullptr;
  size_t scratch_bytes = 0;
  if (kvint2::noalloc_scratch(&scratch, &scratch_bytes) != cudaSuccess) return KV_ERR_CUDA;
  if (pl.bytes > scratch_bytes) return KV_ERR_SCRATCH_LIMIT;
  return cuda_status(kvint2::launch_decode_int2(p, layer, B, q, sink_len, hist_len, recent_len,
                                                recent_start, page_table, max_pages_per_seq, pl,
                                                softmax_scale, out, scratch,
                                                static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_debug_stall_first_copy(kv_pool_t* pool, int32_t enable, int32_t max_polls) {
  if (!pool || max_polls < 0) return KV_ERR_INVALID_ARG;
  // those decodes wait for their copies in flight with the same limit: it has to outlast them
  const int kind = pool->p.cfg.kind;
  if (kind != KV_POOL_FP8 && kind != KV_POOL_FP4 && max_polls > 0 && max_polls < 1024) return KV_ERR_INVALID_ARG;
  pool->p.test_stall_first_copy = enable == 2 ? 2 : enable != 0;
  pool->p.test_wait_polls = max_polls;
  return KV_OK;
}

kv_status_t kv_append_bf16(kv_pool_t* pool, int32_t layer, int32_t n_seqs, const void* k,
                           const void* v, const int32_t* cu_tokens, const int32_t* start_pos,
                           const int32_t* page_table, int32_t max_pages_per_seq,
                           int32_t max_tokens_per_seq, void* stream) {
  if (!valid_layer(pool, layer) || n_seqs < 0 || max_pages_per_seq <= 0 || max_tokens_per_seq < 0)
    return KV_ERR_INVALID_ARG;
  if (pool->p.cfg.kind != KV_POOL_BF16) return KV_ERR_INVALID_ARG;
  if (n_seqs > 0 && (!k || !v || !cu_tokens || !start_pos || !page_table)) return KV_ERR_INVALID_ARG;
  if (((uintptr_t)k & 15) || ((uintptr_t)v & 15)) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_append_bf16(pool->p, layer, n_seqs, k, v, cu_tokens, start_pos,
                                                page_table, max_pages_per_seq, max_tokens_per_seq,
                                                static_cast<cudaStream_t>(stream)));
}

size_t kv_decode_multi_workspace_bytes(const kv_pool_t* pool, int32_t B, int32_t T,
                                       int32_t max_hist_len) {
  if (!pool || B <= 0 || T <= 0 || max_hist_len < 0 || B > pool->p.cfg.max_seqs) return 0;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_INT2_3TIER || !is_pow2_in((int)std::min<int64_t>((int64_t)T * p.G, 16), 1, 8))
    return 0;
  return kvint2::plan_decode_int2(p, B, max_hist_len, T).bytes;
}

kv_status_t kv_decode_attention_multi(kv_pool_t* pool, int32_t layer, int32_t B, int32_t T,
                                      const void* q, const int32_t* sink_len,
                                      const int32_t* hist_len, const int32_t* recent_len,
                                      const int32_t* recent_start, const int32_t* page_table,
                                      int32_t max_pages_per_seq, int32_t max_hist_len,
                                      float softmax_scale, float* out, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_layer(pool, layer) || B <= 0 || T <= 0 || max_pages_per_seq <= 0 || max_hist_len < 0)
    return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_INT2_3TIER || B > p.cfg.max_seqs) return KV_ERR_INVALID_ARG;
  if ((int64_t)T * p.G > 8 || !is_pow2_in(T * p.G, 1, 8)) return KV_ERR_UNSUPPORTED;
  if (!q || !sink_len || !hist_len || !recent_len || !recent_start || !page_table || !out ||
      !workspace)
    return KV_ERR_INVALID_ARG;
  if ((int64_t)max_hist_len > (int64_t)max_pages_per_seq * p.cfg.page_size || max_hist_len > kvint2::kMaxDecodeLen)
    return KV_ERR_INVALID_ARG;
  if (((uintptr_t)workspace & 15) || ((uintptr_t)q & 1) || ((uintptr_t)lse & 3)) return KV_ERR_INVALID_ARG;
  kvint2::DecodePlan pl = kvint2::plan_decode_int2(p, B, max_hist_len, T);
  if (workspace_bytes < pl.bytes) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_decode_int2(p, layer, B, q, sink_len, hist_len, recent_len,
                                                recent_start, page_table, max_pages_per_seq, pl,
                                                softmax_scale, out, workspace,
                                                static_cast<cudaStream_t>(stream), T, lse));
}

static_assert(kvint2::kMaxDecodeLen == KV_MAX_DECODE_LEN, "one decode length bound");

kv_status_t kv_decode_attention_bf16(kv_pool_t* pool, int32_t layer, int32_t B, const void* q,
                                     const int32_t* seq_len, const int32_t* page_table,
                                     int32_t max_pages_per_seq, int32_t max_seq_len,
                                     float softmax_scale, float* out, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (!valid_layer(pool, layer) || B <= 0 || max_pages_per_seq <= 0 || max_seq_len < 0)
    return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_BF16 || B > p.cfg.max_seqs) return KV_ERR_INVALID_ARG;
  if (!q || !seq_len || !page_table || !out || !workspace) return KV_ERR_INVALID_ARG;
  if ((int64_t)max_seq_len > (int64_t)max_pages_per_seq * p.cfg.page_size || max_seq_len > kvint2::kMaxDecodeLen)
    return KV_ERR_INVALID_ARG;
  if (((uintptr_t)workspace & 15) || ((uintptr_t)q & 1)) return KV_ERR_INVALID_ARG;
  kvint2::DecodePlan pl = kvint2::plan_decode_bf16(p, B, max_seq_len);
  if (workspace_bytes < pl.bytes) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_decode_bf16(p, layer, B, q, seq_len, page_table,
                                                max_pages_per_seq, pl, softmax_scale, out,
                                                workspace, static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_pool_get_fp8_layout(const kv_pool_t* pool, int32_t layer, kv_fp8_layout_t* out) {
  if (!valid_layer(pool, layer) || !out || pool->p.cfg.kind != KV_POOL_FP8) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  const size_t per_page = p.cfg.page_size / kvint2::kTile;
  out->codes = pool->fp8.codes + (size_t)layer * pool->fp8.layer_stride;
  out->exps = pool->fp8.exps + (size_t)layer * pool->fp8.exp_layer_stride;
  out->tile_bytes = kvint2::kFp8TileBytes;
  out->codes_layer_stride = pool->fp8.layer_stride;
  out->codes_head_stride = per_page * kvint2::kFp8TileBytes;
  out->codes_page_stride = out->codes_head_stride * p.cfg.num_kv_heads;
  out->exps_layer_stride = pool->fp8.exp_layer_stride;
  out->exps_head_stride = per_page * 2;
  out->exps_page_stride = out->exps_head_stride * p.cfg.num_kv_heads;
  return KV_OK;
}

kv_status_t kv_pool_set_rope(kv_pool_t* pool, int32_t layer, const kv_rope_config_t* cfg) {
  if (!valid_layer(pool, layer) || !cfg) return KV_ERR_INVALID_ARG;
  kvint2::RopeParams r;
  const kv_status_t st = kvint2::rope_params(*cfg, &r);
  if (st == KV_OK) {
    pool->rope[layer] = r;
    pool->axes[layer] = kvint2::RopeAxes{};
  }
  return st;
}

kv_status_t kv_pool_set_rope_axes(kv_pool_t* pool, int32_t layer, int32_t n_axes, const int32_t* axis,
                                  int32_t n_pairs) {
  if (!valid_layer(pool, layer) || !axis || n_axes < 1 || n_axes > 4) return KV_ERR_INVALID_ARG;
  const int pairs = pool->rope[layer].rd / 2;
  if (pairs == 0 || n_pairs != pairs) return KV_ERR_INVALID_ARG;
  kvint2::RopeAxes x{};
  x.n = n_axes;
  for (int i = 0; i < pairs; ++i) {
    if (axis[i] < 0 || axis[i] >= n_axes) return KV_ERR_INVALID_ARG;
    x.axis[i] = (uint8_t)axis[i];
  }
  pool->axes[layer] = x;
  return KV_OK;
}

kv_status_t kv_rope_apply(const kv_pool_t* pool, int32_t layer, int32_t n_tokens, const int32_t* positions,
                          const void* q, int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                          int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  const kvint2::RopeRows rq{q, q_stride, q_out, q_out_stride}, rk{k, k_stride, k_out, k_out_stride};
  if (kv_status_t st = check_rope(pool, layer, n_tokens, positions, rq, rk); st != KV_OK) return st;
  return cuda_status(kvint2::launch_rope(pool->p, pool->rope[layer], n_tokens, positions, rq, rk,
                                         static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_rope_apply_axes(const kv_pool_t* pool, int32_t layer, int32_t n_tokens, const int32_t* positions,
                               int64_t pos_stride, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  const kvint2::RopeRows rq{q, q_stride, q_out, q_out_stride}, rk{k, k_stride, k_out, k_out_stride};
  if (kv_status_t st = check_rope(pool, layer, n_tokens, positions, rq, rk); st != KV_OK) return st;
  if (pos_stride < n_tokens) return KV_ERR_INVALID_ARG;
  return cuda_status(kvint2::launch_rope_axes(pool->p, pool->rope[layer], pool->axes[layer], n_tokens, positions,
                                              pos_stride, rq, rk, static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_append_fp8(kv_pool_t* pool, int32_t layer, int32_t n_seqs, const void* q, int64_t q_stride,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int32_t* cu_tokens, const int32_t* start_pos, const int32_t* page_table,
                          int32_t max_pages_per_seq, int32_t max_tokens_per_seq, void* q_out, void* stream) {
  if (!valid_layer(pool, layer) || n_seqs < 0 || max_pages_per_seq <= 0 || max_tokens_per_seq < 0)
    return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_FP8) return KV_ERR_INVALID_ARG;
  if (n_seqs > 0 && (!k || !v || !cu_tokens || !start_pos || !page_table)) return KV_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return KV_ERR_INVALID_ARG;
  const int Hq = p.cfg.num_q_heads, Hkv = p.cfg.num_kv_heads;
  if (n_seqs > 0 && (!valid_rows(k, k_stride, Hkv) || !valid_rows(v, v_stride, Hkv))) return KV_ERR_INVALID_ARG;
  if (q && (!valid_rows(q, q_stride, Hq) || !aligned16(q_out))) return KV_ERR_INVALID_ARG;
  if (q && q == q_out && q_stride != (int64_t)Hq * 128) return KV_ERR_INVALID_ARG;
  if ((int64_t)n_seqs * (((int64_t)max_tokens_per_seq + 30) / kvint2::kTile) > INT32_MAX) return KV_ERR_INVALID_ARG;
  if (kv_status_t st = on_pool_device(p); st != KV_OK) return st;
  return cuda_status(kvint2::launch_append_fp8(p, pool->fp8, pool->rope[layer], layer, n_seqs,
                                               {q, q_stride, q_out, (int64_t)Hq * 128}, k, k_stride, v, v_stride,
                                               cu_tokens, start_pos, page_table, max_pages_per_seq,
                                               max_tokens_per_seq, static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_decode_attention_fp8(kv_pool_t* pool, int32_t layer, int32_t B, const void* q,
                                    const int32_t* seq_len, const int32_t* page_table, int32_t max_pages_per_seq,
                                    int32_t max_seq_len, float softmax_scale, int32_t window, int32_t n_sink,
                                    void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (kv_status_t st = check_decode(pool, KV_POOL_FP8, layer, B, q, seq_len, page_table, max_pages_per_seq, max_seq_len,
                                    softmax_scale, window, n_sink, out, lse, workspace);
      st != KV_OK)
    return st;
  const Pool& p = pool->p;
  if (workspace_bytes < kvint2::decode_fp8_workspace(p, B, max_seq_len)) return KV_ERR_INVALID_ARG;
  if (kv_status_t st = on_pool_device(p); st != KV_OK) return st;
  return cuda_status(kvint2::launch_decode_fp8(p, pool->fp8, layer, B,
                                               {q, seq_len, page_table, max_pages_per_seq, max_seq_len, softmax_scale,
                                                kvint2::effective_window(window, max_seq_len), n_sink, out, lse,
                                                workspace},
                                               static_cast<cudaStream_t>(stream)));
}

size_t kv_prefill_workspace_bytes(const kv_pool_t* pool, int32_t n_seqs, int32_t max_q_per_seq,
                                  int32_t max_seq_len) {
  if (!pool || pool->p.cfg.kind != KV_POOL_FP8 || !valid_prefill(pool->p, n_seqs, max_q_per_seq) ||
      max_seq_len < 0 || max_seq_len > kvint2::kMaxDecodeLen)
    return 0;
  return kvint2::prefill_fp8_workspace_up_to(pool->p, n_seqs, max_q_per_seq, max_seq_len);
}

kv_status_t kv_prefill_attention_fp8(kv_pool_t* pool, int32_t layer, int32_t n_seqs, const void* q,
                                     const int32_t* cu_q, const int32_t* seq_len, const int32_t* page_table,
                                     int32_t max_pages_per_seq, int32_t max_q_per_seq, int32_t max_seq_len,
                                     float softmax_scale, int32_t window, int32_t n_sink, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_layer(pool, layer) || max_pages_per_seq <= 0 || max_seq_len < 0) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (p.cfg.kind != KV_POOL_FP8 || !valid_prefill(p, n_seqs, max_q_per_seq)) return KV_ERR_INVALID_ARG;
  if (!q || !cu_q || !seq_len || !page_table || !out || !workspace) return KV_ERR_INVALID_ARG;
  if (window < 0 || n_sink < 0 || !std::isfinite(softmax_scale)) return KV_ERR_INVALID_ARG;
  if ((int64_t)max_seq_len > (int64_t)max_pages_per_seq * p.cfg.page_size || max_seq_len > kvint2::kMaxDecodeLen)
    return KV_ERR_INVALID_ARG;
  if (!aligned16(workspace) || !aligned16(q) || !aligned16(out) || ((uintptr_t)lse & 3)) return KV_ERR_INVALID_ARG;
  const size_t need = kvint2::prefill_fp8_workspace(p, n_seqs, max_q_per_seq, max_seq_len);
  if (need == 0 || workspace_bytes < need) return KV_ERR_INVALID_ARG;
  if (kv_status_t st = on_pool_device(p); st != KV_OK) return st;
  return cuda_status(kvint2::launch_prefill_fp8(p, pool->fp8, layer, n_seqs, cu_q, max_q_per_seq,
                                                {q, seq_len, page_table, max_pages_per_seq, max_seq_len, softmax_scale,
                                                 kvint2::effective_window(window, max_seq_len), n_sink, out, lse,
                                                 workspace},
                                                static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_pool_get_fp4_layout(const kv_pool_t* pool, int32_t layer, kv_fp4_layout_t* out) {
  if (!valid_layer(pool, layer) || !out || pool->p.cfg.kind != KV_POOL_FP4) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  out->tiles = pool->fp4.tiles + (size_t)layer * pool->fp4.layer_stride;
  out->tile_bytes = kvint2::kFp4TileBytes;
  out->layer_stride = pool->fp4.layer_stride;
  out->head_stride = (size_t)(p.cfg.page_size / kvint2::kTile) * kvint2::kFp4TileBytes;
  out->page_stride = out->head_stride * p.cfg.num_kv_heads;
  return KV_OK;
}

kv_status_t kv_pool_set_fp4_range(kv_pool_t* pool, int32_t layer, int32_t k_exp, int32_t v_exp) {
  if (!valid_layer(pool, layer) || pool->p.cfg.kind != KV_POOL_FP4) return KV_ERR_INVALID_ARG;
  constexpr int most = kvint2::kFp4ExpMax;
  if (k_exp < -most || k_exp > most || v_exp < -most || v_exp > most) return KV_ERR_INVALID_ARG;
  pool->range[layer] = {k_exp, v_exp};
  return KV_OK;
}

kv_status_t kv_append_fp4(kv_pool_t* pool, int32_t layer, int32_t n_seqs, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* cu_tokens, const int32_t* start_pos,
                          const int32_t* page_table, int32_t max_pages_per_seq, int32_t max_tokens_per_seq,
                          void* stream) {
  if (kv_status_t st = check_fp4_tokens(pool, layer, n_seqs, cu_tokens, start_pos, page_table, max_pages_per_seq,
                                        max_tokens_per_seq);
      st != KV_OK)
    return st;
  const Pool& p = pool->p;
  const int Hkv = p.cfg.num_kv_heads;
  if (n_seqs > 0 && (!k || !v || !valid_rows(k, k_stride, Hkv) || !valid_rows(v, v_stride, Hkv)))
    return KV_ERR_INVALID_ARG;
  if (kv_status_t st = on_pool_device(p); st != KV_OK) return st;
  return cuda_status(kvint2::launch_append_fp4(
      p, kvint2::fp4_layer(p, pool->fp4, pool->range[layer], layer),
      {n_seqs, cu_tokens, start_pos, page_table, max_pages_per_seq, max_tokens_per_seq},
      {const_cast<void*>(k), const_cast<void*>(v), k_stride, v_stride}, static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_read_fp4(const kv_pool_t* pool, int32_t layer, int32_t n_seqs, const int32_t* cu_tokens,
                        const int32_t* start_pos, const int32_t* page_table, int32_t max_pages_per_seq,
                        int32_t max_tokens_per_seq, void* k_out, int64_t k_out_stride, void* v_out,
                        int64_t v_out_stride, void* stream) {
  if (kv_status_t st = check_fp4_tokens(pool, layer, n_seqs, cu_tokens, start_pos, page_table, max_pages_per_seq,
                                        max_tokens_per_seq);
      st != KV_OK)
    return st;
  const Pool& p = pool->p;
  const int Hkv = p.cfg.num_kv_heads;
  if (n_seqs > 0 && !k_out && !v_out) return KV_ERR_INVALID_ARG;
  if ((k_out && !valid_rows(k_out, k_out_stride, Hkv)) || (v_out && !valid_rows(v_out, v_out_stride, Hkv)))
    return KV_ERR_INVALID_ARG;
  if (kv_status_t st = on_pool_device(p); st != KV_OK) return st;
  return cuda_status(kvint2::launch_read_fp4(p, kvint2::fp4_layer(p, pool->fp4, pool->range[layer], layer),
                                             {n_seqs, cu_tokens, start_pos, page_table, max_pages_per_seq,
                                              max_tokens_per_seq},
                                             {k_out, v_out, k_out_stride, v_out_stride},
                                             static_cast<cudaStream_t>(stream)));
}

kv_status_t kv_decode_attention_fp4(kv_pool_t* pool, int32_t layer, int32_t B, const void* q,
                                    const int32_t* seq_len, const int32_t* page_table, int32_t max_pages_per_seq,
                                    int32_t max_seq_len, float softmax_scale, int32_t window, int32_t n_sink,
                                    void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (kv_status_t st = check_decode(pool, KV_POOL_FP4, layer, B, q, seq_len, page_table, max_pages_per_seq, max_seq_len,
                                    softmax_scale, window, n_sink, out, lse, workspace);
      st != KV_OK)
    return st;
  const Pool& p = pool->p;
  const int seen = kvint2::effective_window(window, max_seq_len);
  const int splits = kvint2::decode_fp4_splits(p, B, max_seq_len, seen, n_sink);
  if (workspace_bytes < kvint2::decode_fp4_workspace(p, B, splits)) return KV_ERR_INVALID_ARG;
  if (kv_status_t st = on_pool_device(p); st != KV_OK) return st;
  return cuda_status(kvint2::launch_decode_fp4(p, kvint2::fp4_layer(p, pool->fp4, pool->range[layer], layer), layer, B,
                                               splits,
                                               {q, seq_len, page_table, max_pages_per_seq, max_seq_len, softmax_scale,
                                                seen, n_sink, out, lse, workspace},
                                               static_cast<cudaStream_t>(stream)));
}

size_t kv_prompt_workspace_bytes(const kv_pool_t* pool, int32_t n_seqs, int32_t max_q_per_seq, int32_t max_k_per_seq) {
  if (!pool || !valid_prompt(pool->p, n_seqs, max_q_per_seq, max_k_per_seq)) return 0;
  return kvint2::prompt_workspace_up_to(pool->p, n_seqs, max_q_per_seq, max_k_per_seq);
}

kv_status_t kv_prompt_attention(kv_pool_t* pool, int32_t n_seqs, const void* q, int64_t q_stride, int64_t q_rows,
                                const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t kv_rows,
                                const int32_t* cu_q, const int32_t* cu_k, int32_t max_q_per_seq,
                                int32_t max_k_per_seq, float softmax_scale, int32_t window, int32_t n_sink, void* out,
                                float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!pool || !valid_prompt(pool->p, n_seqs, max_q_per_seq, max_k_per_seq)) return KV_ERR_INVALID_ARG;
  const Pool& p = pool->p;
  if (!q || !k || !v || !cu_q || !cu_k || !out || !workspace) return KV_ERR_INVALID_ARG;
  if (q_rows < 0 || q_rows > INT32_MAX || kv_rows < 1 || kv_rows > INT32_MAX) return KV_ERR_INVALID_ARG;
  const int Hkv = p.cfg.num_kv_heads;
  if (!valid_rows(q, q_stride, p.cfg.num_q_heads) || !valid_rows(k, k_stride, Hkv) || !valid_rows(v, v_stride, Hkv))
    return KV_ERR_INVALID_ARG;
  if (q_stride > INT32_MAX || k_stride > INT32_MAX || v_stride > INT32_MAX) return KV_ERR_INVALID_ARG;
  if (window < 0 || n_sink < 0 || !std::isfinite(softmax_scale)) return KV_ERR_INVALID_ARG;
  if (!aligned16(workspace) || !aligned16(out) || ((uintptr_t)lse & 3)) return KV_ERR_INVALID_ARG;
  if (workspace_bytes < kvint2::prompt_workspace(p, n_seqs, max_q_per_seq, max_k_per_seq)) return KV_ERR_INVALID_ARG;
  if (kv_status_t st = on_pool_device(p); st != KV_OK) return st;
  return cuda_status(kvint2::launch_prompt(p,
                                           {q, k, v, q_stride, k_stride, v_stride, q_rows, kv_rows, cu_q, cu_k, n_seqs,
                                            max_q_per_seq, max_k_per_seq, softmax_scale,
                                            kvint2::effective_window(window, max_k_per_seq), n_sink, out, lse, workspace},
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
