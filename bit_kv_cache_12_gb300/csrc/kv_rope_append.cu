// Rotary positions and the append into the 8-bit cache.
//
// Rotation: the pair (a, b) of a head at position p becomes
//   (a cos - b sin, b cos + a sin) * att,  angle = p * w_i,
// in fp32, rounded once (bf16 for q and k rows, e4m3 for cached K).  The angle
// is formed as a fraction of a turn in 64-bit integers, p * (w_i / 2 pi) modulo
// one turn: the product wraps by itself, so the reduction is exact at any
// position and costs one integer multiply; sincospif then sees [-1, 1).
//
// Append: e = the smallest exponent whose range (448 * 2^e) holds the 16 x 128
// values of a tile, codes = e4m3(value * 2^-e).  The K exponent goes by the
// lengths of the rotated pairs, which rotation keeps: it depends on the input
// alone (not on rounding of sines), and the raw bf16 rows give it before the
// first sine is needed.
//
// Bound: memory traffic (2 B in, 1 or 2 B out per channel) for long prompts,
// latency for single tokens.  One CTA owns one 16-token tile of one sequence
// for a slice of the heads: the 16 x 64 cosines and sines are formed once per
// CTA in shared memory and used by every head, and a warp owns the whole
// (tile, head) it quantizes, so the tile's maximum is one warp reduction, no
// atomics, and a tile that already holds tokens has one writer.
#include <cuda_fp8.h>

#include <cmath>

#include "kv_device.cuh"
#include "kv_fp8.h"

namespace kvint2 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// cos / sin rows: 16 pairs (128 B) and 16 B of padding, so that the four runs
// of a token a quarter warp reads fall in different banks
constexpr int kRunStride = 18;                 // float2
constexpr int kTokStride = 4 * kRunStride;     // float2

__device__ __forceinline__ void bf16x2_unpack(uint32_t w, float& a, float& b) {
  a = bf16lo(w);
  b = bf16hi(w);
}

__device__ __forceinline__ uint32_t bf16x2_pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// cos and sin of `turns` (units of 2^-64 of a turn), times att.  The nearest
// quarter turn is taken off in integers, so the fp32 argument is at most a
// quarter of pi and its rounding moves the angle by at most 2^-26.
__device__ __forceinline__ float2 turn_cos_sin(unsigned long long turns, float att) {
  const unsigned long long quarter = (turns + (1ull << 61)) >> 62;
  const int r = (int)((long long)(turns - (quarter << 62)) >> 30);   // in 2^-34 of a turn
  float s, c;
  sincospif((float)r * 0x1p-33f, &s, &c);
  const float x = (quarter & 1) ? -s : c, y = (quarter & 1) ? c : s;
  return (quarter & 2) ? make_float2(-x * att, -y * att) : make_float2(x * att, y * att);
}

// Table of the CTA's 16 tokens: pos < 0 marks a token without work.
__device__ __forceinline__ void fill_table(float2* tab, const RopeParams& rp, const int* pos) {
  const int n = rp.rd >> 1;
  for (int i = threadIdx.x; i < kTile * 64; i += kThreads) {
    const int t = i >> 6, f = i & 63;
    if (f < n && pos[t] >= 0)
      tab[t * kTokStride + (f >> 4) * kRunStride + (f & 15)] =
          turn_cos_sin((unsigned long long)pos[t] * rp.turn[f], rp.att);
  }
}

// 16 channels of a row (run c of 8).
struct Run {
  uint32_t own[8];
};

// read once by this kernel (and perhaps written by it: not the read-only path)
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void load_run(Run& r, const uint16_t* row, int c, bool live) {
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (live) {
    a = ld_once(row + 16 * c);
    b = ld_once(row + 16 * c + 8);
  }
  r.own[0] = a.x; r.own[1] = a.y; r.own[2] = a.z; r.own[3] = a.w;
  r.own[4] = b.x; r.own[5] = b.y; r.own[6] = b.z; r.own[7] = b.w;
}

// The run that channel run c is paired with (half style) sits in another lane of
// the same row (lanes 8k .. 8k + 7).  It is fetched where it is used, twice for a
// quantized tile: kept, it would cost 32 registers and a third of the warps.
__device__ __forceinline__ int mate_lane(const RopeParams& rp, int lane) {
  const int c = lane & 7, n = rp.rd >> 4, h = n >> 1;   // rotated runs, half of them
  return (lane & 24) | (c < h ? c + h : (c < n ? c - h : c));
}
template <bool kPairs>
__device__ __forceinline__ void fetch_mate(const Run& r, uint32_t (&mate)[8], int src) {
  if (!kPairs) {                               // else the pair is in the run itself
#pragma unroll
    for (int i = 0; i < 8; ++i) mate[i] = __shfl_sync(0xffffffffu, r.own[i], src);
  }
}

// The rotated values of the run.
template <bool kPairs>
__device__ __forceinline__ void rotate_run(const Run& r, const uint32_t (&mate)[8], const RopeParams& rp,
                                           const float2* tok, int c, float (&y)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) bf16x2_unpack(r.own[i], y[2 * i], y[2 * i + 1]);
  const int n = rp.rd >> 4;
  if (c >= n) return;
  if (kPairs) {
    const float2* cs = tok + (c >> 1) * kRunStride + (c & 1) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = cs[i];
      const float a = y[2 * i], b = y[2 * i + 1];
      y[2 * i] = a * t.x - b * t.y;
      y[2 * i + 1] = b * t.x + a * t.y;
    }
  } else {
    const int h = n >> 1;
    const float2* cs = tok + (c < h ? c : c - h) * kRunStride;
    const float sg = c < h ? -1.f : 1.f;       // first of the pair: a cos - b sin
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m0, m1;
      bf16x2_unpack(mate[i], m0, m1);
      const float2 t0 = cs[2 * i], t1 = cs[2 * i + 1];
      y[2 * i] = y[2 * i] * t0.x + sg * m0 * t0.y;
      y[2 * i + 1] = y[2 * i + 1] * t1.x + sg * m1 * t1.y;
    }
  }
}

// The largest square the run contributes to the K exponent: pair lengths where
// rotated, magnitudes elsewhere.  Squares of bf16 values are exact in fp32 and
// their sum is rounded once, so every lane and order gives the same value.
template <bool kPairs>
__device__ __forceinline__ float run_square(const Run& r, const uint32_t (&mate)[8], const RopeParams& rp, int c,
                                            bool rotate) {
  const int n = rotate ? rp.rd >> 4 : 0;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    bf16x2_unpack(r.own[i], a, b);
    if (c >= n) {
      m = fmaxf(m, fmaxf(a * a, b * b));
    } else if (kPairs) {
      m = fmaxf(m, fmaf(a, a, b * b));
    } else {
      float ma, mb;
      bf16x2_unpack(mate[i], ma, mb);
      m = fmaxf(m, fmaxf(fmaf(a, a, ma * ma), fmaf(b, b, mb * mb)));
    }
  }
  return (c < n && rp.att2 != 1.f) ? m * rp.att2 : m;
}

__device__ __forceinline__ bool run_nonfinite(const Run& r) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    bad = bad || (r.own[i] & 0x7F80u) == 0x7F80u || (r.own[i] & 0x7F800000u) == 0x7F800000u;
  return bad;
}

// The smallest e with square <= (448 * 2^e)^2 = 1.53125 * 2^(17 + 2e), clamped.
__device__ __forceinline__ int tile_exponent(float square) {
  const uint32_t u = __float_as_uint(square);
  const int k = (int)(u >> 23) - 127;
  if (k == 128) return KV_FP8_EXP_MAX;
  const int e = (k - 16 + ((u & 0x7FFFFFu) > 0x440000u ? 1 : 0)) >> 1;
  return min(max(e, KV_FP8_EXP_MIN), KV_FP8_EXP_MAX);
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Four codes times `f`, rounded back to codes.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
  return e4m3x4(x.x * f, x.y * f, y.x * f, y.y * f);
}

// Byte offset of run c (16 channels) of token t in the stored K or V codes.
__device__ __forceinline__ int code_offset(int tensor, int t, int c) {
  return tensor == 0 ? (t >> 3) * 1024 + (c >> 2) * 512 + (t & 7) * 64 + (c & 3) * 16
                     : ((t & 1) + 2 * (t >> 3)) * 512 + c * 64 + ((t & 7) >> 1) * 16;
}

// One head of 16 tokens, rotated (or not) and stored as bf16: lanes 8k .. 8k+7
// hold one row, four rows per pass.  pos[t] < 0: the row is not touched.
template <bool kPairs>
__device__ __forceinline__ void rows_unit(const RopeParams& rp, const float2* tab, const int* pos, const uint16_t* in,
                                          int64_t in_stride, uint16_t* out, int64_t out_stride, int lane) {
  const int c = lane & 7, src = mate_lane(rp, lane);
  Run r[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    load_run(r[u], in + t * in_stride, c, pos[t] >= 0);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    uint32_t mate[8];
    fetch_mate<kPairs>(r[u], mate, src);
    if (pos[t] < 0) continue;
    float y[16];
    rotate_run<kPairs>(r[u], mate, rp, tab + t * kTokStride, c, y);
    uint4* o = reinterpret_cast<uint4*>(out + t * out_stride + 16 * c);
    o[0] = make_uint4(bf16x2_pack(y[0], y[1]), bf16x2_pack(y[2], y[3]), bf16x2_pack(y[4], y[5]),
                      bf16x2_pack(y[6], y[7]));
    o[1] = make_uint4(bf16x2_pack(y[8], y[9]), bf16x2_pack(y[10], y[11]), bf16x2_pack(y[12], y[13]),
                      bf16x2_pack(y[14], y[15]));
  }
}

struct RopeArgs {
  const uint16_t* in[2];       // q, k
  uint16_t* out[2];
  int64_t in_stride[2], out_stride[2];
  int heads[2];                // 0 where absent
  const int32_t* positions;
  int n_tokens;
};

// kPairs: rotated pairs are neighbouring channels (interleaved style)
template <bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(RopeArgs a, const __grid_constant__ RopeParams rp) {
  __shared__ float2 tab[kTile * kTokStride];
  __shared__ int pos[kTile];
  const int t0 = blockIdx.x * kTile;
  if (threadIdx.x < kTile) pos[threadIdx.x] = t0 + (int)threadIdx.x < a.n_tokens ? a.positions[t0 + threadIdx.x] : -1;
  __syncthreads();
  fill_table(tab, rp, pos);
  __syncthreads();
  const int lane = threadIdx.x & 31, units = a.heads[0] + a.heads[1];
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.y * kWarps) {
    const bool k = u >= a.heads[0];
    const int h = u - (k ? a.heads[0] : 0);
    const int64_t is = k ? a.in_stride[1] : a.in_stride[0], os = k ? a.out_stride[1] : a.out_stride[0];
    rows_unit<kPairs>(rp, tab, pos, (k ? a.in[1] : a.in[0]) + t0 * is + h * 128, is,
                      (k ? a.out[1] : a.out[0]) + t0 * os + h * 128, os, lane);
  }
}

struct AppendFp8Args {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, qo_stride;
  uint16_t* q_out;
  const int32_t *cu, *start, *pt;
  uint8_t* codes;
  int8_t* exps;
  long long num_pages;
  int max_pages, max_tokens, tiles, Hq, Hkv, P;
  int* err;
};

// One (tile, head) of K (tensor 0) or V (tensor 1): tokens [t0, t1) of the tile
// are new, in + t * stride is the row of tile slot t.
template <bool kPairs>
__device__ __forceinline__ void quant_unit(const RopeParams& rp, const float2* tab, const uint16_t* in, int64_t stride,
                                           int t0, int t1, int tensor, uint8_t* codes, int8_t* exp, int lane) {
  const int c = lane & 7, src = mate_lane(rp, lane);
  const bool rot = tensor == 0;
  const int e_old = t0 > 0 ? *exp : KV_FP8_EXP_MIN;
  Run r[4];
  uint32_t bad = 0;
  float sq = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    load_run(r[u], in + t * stride, c, t >= t0 && t < t1);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t mate[8];
    if (rot) fetch_mate<kPairs>(r[u], mate, src);
    const uint32_t b = __ballot_sync(0xffffffffu, run_nonfinite(r[u]));
    if ((b >> (lane & 24)) & 0xFFu)
      bad |= 1u << u;
    else
      sq = fmaxf(sq, run_square<kPairs>(r[u], mate, rp, c, rot));
  }
  const int e = max(tile_exponent(warp_max_xor(sq, 1)), e_old);
  if (t0 > 0 && e > e_old) {                     // earlier tokens move to the larger exponent
    const float f = pow2i(max(e_old - e, -126));
    for (int t = lane >> 3; t < t0; t += 4) {
      uint4* p = reinterpret_cast<uint4*>(codes + code_offset(tensor, t, c));
      uint4 w = *p;
      w.x = rescale4(w.x, f);
      w.y = rescale4(w.y, f);
      w.z = rescale4(w.z, f);
      w.w = rescale4(w.w, f);
      *p = w;
    }
  }
  const float inv = pow2i(-e);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    uint32_t mate[8];
    if (rot) fetch_mate<kPairs>(r[u], mate, src);
    if (t < t0 || t >= t1) continue;
    uint4 w = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (!((bad >> u) & 1)) {
      float y[16];
      if (rot) {
        rotate_run<kPairs>(r[u], mate, rp, tab + t * kTokStride, c, y);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) bf16x2_unpack(r[u].own[i], y[2 * i], y[2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] *= inv;
      w = make_uint4(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]),
                     e4m3x4(y[8], y[9], y[10], y[11]), e4m3x4(y[12], y[13], y[14], y[15]));
    }
    *reinterpret_cast<uint4*>(codes + code_offset(tensor, t, c)) = w;
  }
  if (lane == 0 && (t0 == 0 || e > e_old)) *exp = (int8_t)e;
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads, 3) append_fp8_kernel(AppendFp8Args a, const __grid_constant__ RopeParams rp) {
  __shared__ float2 tab[kTile * kTokStride];
  __shared__ int pos[kTile];
  const int s = blockIdx.x / a.tiles, i = blockIdx.x - s * a.tiles;
  const int c0 = a.cu[s];
  int n = a.cu[s + 1] - c0;
  const int start = a.start[s];
  if (n < 0 || n > a.max_tokens) {
    if (i == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    n = min(n, a.max_tokens);
  }
  if (n <= 0) return;
  if (start < 0 || (long long)start + n > (long long)a.max_pages * a.P) {
    if (i == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return;
  }
  // tile slots [t0, t1) of the i-th tile the sequence's new tokens touch
  const long long base = ((long long)(start / kTile) + i) * kTile;   // position of slot 0
  const long long lo = max(base, (long long)start), hi = min(base + kTile, (long long)start + n);
  if (lo >= hi) return;
  const int t0 = (int)(lo - base), t1 = (int)(hi - base);
  if (threadIdx.x < kTile) {
    const bool in = (int)threadIdx.x >= t0 && (int)threadIdx.x < t1;
    pos[threadIdx.x] = in ? (int)(base + threadIdx.x) : -1;
  }
  __syncthreads();
  fill_table(tab, rp, pos);
  const int pid = a.pt[(size_t)s * a.max_pages + base / a.P];
  const bool page_ok = pid >= 0 && pid < a.num_pages;
  if (!page_ok && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_PAGE_ID);
  __syncthreads();
  const int lane = threadIdx.x & 31, nkv = 2 * a.Hkv, units = nkv + (a.q ? a.Hq : 0);
  const int per = a.P / kTile, sub = (int)(base / kTile % per);
  const int64_t row0 = (int64_t)c0 + (base - start);       // input row of slot 0 (rows t0 .. t1 - 1 exist)
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.y * kWarps) {
    if (u < nkv) {
      if (!page_ok) continue;
      const int tensor = u >= a.Hkv, h = u - (tensor ? a.Hkv : 0);
      const size_t tile = ((size_t)pid * a.Hkv + h) * per + sub;
      const int64_t stride = tensor ? a.v_stride : a.k_stride;
      quant_unit<kPairs>(rp, tab, (tensor ? a.v : a.k) + row0 * stride + h * 128, stride, t0, t1, tensor,
                 a.codes + tile * kFp8TileBytes + tensor * 2048, a.exps + tile * 2 + tensor, lane);
    } else {
      const int h = u - nkv;
      rows_unit<kPairs>(rp, tab, pos, a.q + row0 * a.q_stride + h * 128, a.q_stride, a.q_out + row0 * a.qo_stride + h * 128,
                a.qo_stride, lane);
    }
  }
}

// Slices of the heads per tile: enough CTAs for four per SM, at most one unit
// per warp.
unsigned slices(const Pool& p, long long tiles, int units) {
  const long long want = (4ll * p.sm_count + tiles - 1) / tiles;
  return (unsigned)std::max(1ll, std::min<long long>((units + kWarps - 1) / kWarps, want));
}

}  // namespace

kv_status_t rope_params(const kv_rope_config_t& c, RopeParams* out) {
  RopeParams r{};
  const int d = c.rotary_dim;
  if (d < 0 || d > 128) return KV_ERR_INVALID_ARG;
  if (d % 32) return KV_ERR_UNSUPPORTED;
  if (c.style != KV_ROPE_HALF && c.style != KV_ROPE_INTERLEAVED) return KV_ERR_INVALID_ARG;
  if (c.scaling < KV_ROPE_SCALE_NONE || c.scaling > KV_ROPE_SCALE_YARN) return KV_ERR_INVALID_ARG;
  if (!(c.attention_factor >= 0) || !std::isfinite(c.attention_factor)) return KV_ERR_INVALID_ARG;
  double att = c.attention_factor;
  double w[64] = {};
  if (d > 0 && c.inv_freq) {
    for (int i = 0; i < d / 2; ++i) {
      w[i] = c.inv_freq[i];
      if (!std::isfinite(w[i])) return KV_ERR_INVALID_ARG;
    }
  } else if (d > 0) {
    double base = c.theta;
    if (!std::isfinite(base) || !(base > 1)) return KV_ERR_INVALID_ARG;
    if (c.scaling != KV_ROPE_SCALE_NONE && (!std::isfinite(c.factor) || !(c.factor >= 1))) return KV_ERR_INVALID_ARG;
    if (c.scaling == KV_ROPE_SCALE_NTK) base *= std::pow(c.factor, (double)d / (d - 2));
    for (int i = 0; i < d / 2; ++i) w[i] = std::pow(base, -2.0 * i / d);
    if (c.scaling == KV_ROPE_SCALE_LINEAR)
      for (int i = 0; i < d / 2; ++i) w[i] /= c.factor;
    if (c.scaling == KV_ROPE_SCALE_YARN) {
      const double fast = c.beta_fast == 0 ? 32.0 : c.beta_fast, slow = c.beta_slow == 0 ? 1.0 : c.beta_slow;
      if (c.original_max_position <= 0 || !(slow > 0) || !(fast > slow) || !std::isfinite(fast))
        return KV_ERR_INVALID_ARG;
      // the pair index that makes `turns` turns over the trained context
      auto index = [&](double turns) {
        return d * std::log(c.original_max_position / (turns * 2 * M_PI)) / (2 * std::log(base));
      };
      const double low = std::max(std::floor(index(fast)), 0.0);
      const double high = std::min(std::ceil(index(slow)), (double)(d - 1));
      for (int i = 0; i < d / 2; ++i) {
        const double ramp = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
        w[i] = w[i] / c.factor * ramp + w[i] * (1.0 - ramp);
      }
      if (att == 0) att = 0.1 * std::log(c.factor) + 1.0;
    }
  }
  r.rd = d;
  r.interleaved = c.style == KV_ROPE_INTERLEAVED;
  r.att = (float)(att == 0 ? 1.0 : att);
  r.att2 = (float)((double)r.att * (double)r.att);
  for (int i = 0; i < d / 2; ++i) {
    double f = w[i] / (2 * M_PI);
    f -= std::floor(f);                          // [0, 1]: turns per position modulo one turn
    const double hi = std::floor(std::ldexp(f, 32)), lo = std::ldexp(f, 64) - std::ldexp(hi, 32);
    r.turn[i] = ((unsigned long long)hi << 32) + (unsigned long long)lo;
  }
  *out = r;
  return KV_OK;
}

cudaError_t launch_rope(const Pool& p, const RopeParams& r, int n_tokens, const int32_t* positions, const RopeRows& q,
                        const RopeRows& k, cudaStream_t s) {
  if (n_tokens == 0) return cudaSuccess;
  RopeArgs a{};
  const RopeRows* rows[2] = {&q, &k};
  for (int w = 0; w < 2; ++w) {
    a.in[w] = static_cast<const uint16_t*>(rows[w]->in);
    a.out[w] = static_cast<uint16_t*>(rows[w]->out);
    a.in_stride[w] = rows[w]->in_stride;
    a.out_stride[w] = rows[w]->out_stride;
    a.heads[w] = rows[w]->in ? (w ? p.cfg.num_kv_heads : p.cfg.num_q_heads) : 0;
  }
  a.positions = positions;
  a.n_tokens = n_tokens;
  const long long tiles = ((long long)n_tokens + kTile - 1) / kTile;
  const dim3 grid((unsigned)tiles, slices(p, tiles, a.heads[0] + a.heads[1]));
  if (r.interleaved)
    rope_kernel<true><<<grid, kThreads, 0, s>>>(a, r);
  else
    rope_kernel<false><<<grid, kThreads, 0, s>>>(a, r);
  return cudaGetLastError();
}

cudaError_t launch_append_fp8(const Pool& p, const Fp8Store& f, const RopeParams& r, int layer, int n_seqs,
                              const RopeRows& q, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* cu, const int32_t* start, const int32_t* pt, int max_pages,
                              int max_tokens, cudaStream_t s) {
  if (n_seqs == 0 || max_tokens == 0) return cudaSuccess;
  AppendFp8Args a{};
  a.q = static_cast<const uint16_t*>(q.in);
  a.q_stride = q.in_stride;
  a.q_out = static_cast<uint16_t*>(q.out);
  a.qo_stride = q.out_stride;
  a.k = static_cast<const uint16_t*>(k);
  a.k_stride = k_stride;
  a.v = static_cast<const uint16_t*>(v);
  a.v_stride = v_stride;
  a.cu = cu;
  a.start = start;
  a.pt = pt;
  a.codes = f.codes + (size_t)layer * f.layer_stride;
  a.exps = f.exps + (size_t)layer * f.exp_layer_stride;
  a.num_pages = p.cfg.num_pages;
  a.max_pages = max_pages;
  a.max_tokens = max_tokens;
  a.tiles = (int)(((long long)max_tokens + 30) / kTile);   // n tokens touch at most this many tiles
  a.Hq = p.cfg.num_q_heads;
  a.Hkv = p.cfg.num_kv_heads;
  a.P = p.cfg.page_size;
  a.err = p.err;
  const long long tiles = (long long)n_seqs * a.tiles;
  const dim3 grid((unsigned)tiles, slices(p, tiles, 2 * a.Hkv + (a.q ? a.Hq : 0)));
  if (r.interleaved)
    append_fp8_kernel<true><<<grid, kThreads, 0, s>>>(a, r);
  else
    append_fp8_kernel<false><<<grid, kThreads, 0, s>>>(a, r);
  return cudaGetLastError();
}

}  // namespace kvint2
