// Rotary positions and the append into the 8-bit cache.
//
// Rotation: the pair (a, b) of a head at position p becomes
//   (a cos - b sin, b cos + a sin) * att,  angle = p * w_i,
// in fp32, rounded once (bf16 for q and k rows, e4m3 for cached K).  The angle
// is formed as a fraction of a turn in 64-bit integers, p * (w_i / 2 pi) modulo
// one turn: the product wraps by itself, so the reduction costs one integer
// multiply and adds nothing to the speed's own 2^-65 of a turn per position;
// sincospif then sees an eighth of a turn to either side.
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
// atomics, and a tile that already holds tokens has one writer.  A lane holds
// both members of its pairs (two chunks of eight channels), so nothing crosses
// lanes but the maximum.  What counted for a prompt of 8192 tokens (32 query heads,
// 8 KV heads): registers (180 -> 80, one -> three CTAs per SM: 76 -> 47 us),
// instructions (pairs in a lane, paired arithmetic), now with 64 registers and four
// CTAs (39; the append spills 12 to 24 bytes for it), starting before the kernel in front has ended
// (37.3), rows on their way while the table is formed or the unit before is worked
// on (35.0 us, 5.3 TB/s: 0.79 of a plain copy; issue slots half in use).  Rotary
// rows alone, 8192 tokens of 64 + 8 heads: 50.7 us, 6.0 TB/s, 0.89 of a plain copy
// (54 to 57 with such prefetches; with a warp's first rows in registers before the
// table is formed 50.7 instead of 52).
#include <cuda_fp8.h>

#include <cmath>

#include "kv_device.cuh"
#include "kv_fp4.h"

namespace kvint2 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Cosines and sines of a token: pair i = 8 l + e (lane l of the token's eight)
// at 4 l + e % 4 + 32 (e / 4), the sines 64 behind; 4 floats of padding.  The
// eight lanes of a token read 16 bytes each, all banks once.
constexpr int kTokStride = 132;

__device__ __forceinline__ uint32_t bf16x2_pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pairs of fp32 values in one register pair: one instruction for both, each
// rounded as the scalar one.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// cos and sin of `turns` (units of 2^-64 of a turn), times att.  The nearest
// quarter turn is taken off in integers, so the fp32 argument is at most an eighth
// of a turn and its rounding moves the angle by at most 2^-28 of a turn (2^-25.3
// radians), and by less the nearer it is to a quarter.
__device__ __forceinline__ float2 turn_cos_sin(unsigned long long turns, float att) {
  const unsigned long long quarter = (turns + (1ull << 61)) >> 62;
  const int r = (int)((long long)(turns - (quarter << 62)) >> 30);   // in 2^-34 of a turn
  float s, c;
  sincospif((float)r * 0x1p-33f, &s, &c);
  const float x = (quarter & 1) ? -s : c, y = (quarter & 1) ? c : s;
  return (quarter & 2) ? make_float2(-x * att, -y * att) : make_float2(x * att, y * att);
}

// Table of the CTA's 16 tokens: pos < 0 marks a token without work.
__device__ __forceinline__ void fill_table(float* tab, const RopeParams& rp, const int* pos) {
  const int n = rp.rd >> 1;
  for (int i = threadIdx.x; i < kTile * 64; i += kThreads) {
    const int t = i >> 6, f = i & 63;
    if (f < n && pos[t] >= 0) {
      const float2 cs = turn_cos_sin((unsigned long long)pos[t] * rp.turn[f], rp.att);
      float* d = tab + t * kTokStride + 4 * (f >> 3) + (f & 3) + 32 * ((f >> 2) & 1);
      d[0] = cs.x;
      d[64] = cs.y;
    }
  }
}

// The 16 channels of a row that a lane holds: two chunks of eight.  Half style:
// the first and the second members of eight pairs where rotated, else two
// neighbouring chunks.  Interleaved (kPairs): neighbouring chunks, the pairs in
// their words.  No value crosses lanes.
struct Chunks {
  int a, b;                                    // first channels
  bool rotated;
};
template <bool kPairs>
__device__ __forceinline__ Chunks chunks_of(const RopeParams& rp, int lane) {
  const int l = lane & 7;
  if (kPairs) return {16 * l, 16 * l + 8, 16 * l < rp.rd};
  const int np = rp.rd >> 4;                   // lanes that hold pairs
  return l < np ? Chunks{8 * l, 8 * l + (rp.rd >> 1), true} : Chunks{16 * l, 16 * l + 8, false};
}

// read once by this kernel (and perhaps written by it: not the read-only path)
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

struct Run {
  uint32_t w[8];                               // chunk a, chunk b
};

__device__ __forceinline__ void load_run(Run& r, const uint16_t* row, int a, int b, bool live) {
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  if (live) {
    x = ld_once(row + a);
    y = ld_once(row + b);
  }
  r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
  r.w[4] = y.x; r.w[5] = y.y; r.w[6] = y.z; r.w[7] = y.w;
}

__device__ __forceinline__ uint64_t f2_of(uint32_t w) { return f2(bf16lo(w), bf16hi(w)); }

// The rotated values, chunk a then chunk b, as fp32 pairs.  kScaled: of the row times
// `scale` (a pair of the same power of two).
template <bool kPairs, bool kScaled>
__device__ __forceinline__ void rotate_run(const Run& r, uint64_t scale, const float* tok, int lane, bool rotated,
                                           uint64_t (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = kScaled ? f2_mul(f2_of(r.w[i]), scale) : f2_of(r.w[i]);
  if (!rotated) return;
  const float4* t = reinterpret_cast<const float4*>(tok) + (lane & 7);
  const float4 c0 = t[0], c1 = t[8], s0 = t[16], s1 = t[24];
  if (kPairs) {
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      f2_split(y[i], a, b);
      y[i] = f2(a * c[i] - b * s[i], b * c[i] + a * s[i]);
    }
  } else {
    const uint64_t c[4] = {f2(c0.x, c0.y), f2(c0.z, c0.w), f2(c1.x, c1.y), f2(c1.z, c1.w)};
    const uint64_t s[4] = {f2(s0.x, s0.y), f2(s0.z, s0.w), f2(s1.x, s1.y), f2(s1.z, s1.w)};
    const uint64_t minus = f2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = y[i], b = y[4 + i];
      y[i] = f2_fma(f2_mul(b, minus), s[i], f2_mul(a, c[i]));
      y[4 + i] = f2_fma(a, s[i], f2_mul(b, c[i]));
    }
  }
}

// The largest square the run contributes to the K exponent: pair lengths where
// rotated, magnitudes elsewhere.  Squares of bf16 values are exact in fp32 and
// their sum is rounded once, so every order gives the same value.
template <bool kPairs>
__device__ __forceinline__ float run_square(const Run& r, const RopeParams& rp, bool rotated) {
  float m = 0.f;
  if (kPairs || !rotated) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = bf16lo(r.w[i]), b = bf16hi(r.w[i]);
      m = rotated ? fmaxf(m, fmaf(a, a, b * b)) : fmaxf(m, fmaxf(a * a, b * b));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = f2_of(r.w[i]), b = f2_of(r.w[4 + i]);
      float x, y;
      f2_split(f2_fma(a, a, f2_mul(b, b)), x, y);
      m = fmaxf(m, fmaxf(x, y));
    }
  }
  return rotated && rp.att2 != 1.f ? m * rp.att2 : m;
}

// The largest magnitude of the run, as bf16 bits (above 0x7F7F: not finite).
__device__ __forceinline__ uint32_t run_magnitude(const Run& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, r.w[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}

// The smallest e with square <= (448 * 2^e)^2 = 1.53125 * 2^(17 + 2e), clamped.
__device__ __forceinline__ int tile_exponent(float square) {
  const uint32_t u = __float_as_uint(square);
  const int k = (int)(u >> 23) - 127;
  if (k == 128) return KV_FP8_EXP_MAX;
  const int e = (k - 16 + ((u & 0x7FFFFFu) > 0x440000u ? 1 : 0)) >> 1;
  return min(max(e, KV_FP8_EXP_MIN), KV_FP8_EXP_MAX);
}

// The same from the largest magnitude, as finite bf16 bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ int magnitude_exponent(uint32_t bits) {
  const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 0x7Fu) > 0x60u ? 1 : 0);
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

// Byte offset of channel c (a multiple of 8) of token t in the stored K or V codes.
__device__ __forceinline__ int code_offset(bool v, int t, int c) {
  return v ? ((t & 1) + 2 * (t >> 3)) * 512 + (c >> 4) * 64 + ((t & 7) >> 1) * 16 + (c & 15)
           : (t >> 3) * 1024 + (c >> 6) * 512 + (t & 7) * 64 + (c & 63);
}

// One head of 16 tokens, rotated and stored as bf16: lanes 8k .. 8k + 7 hold one
// row, four rows per pass.  pos[t] < 0: the row is not touched.
template <bool kPairs>
__device__ __forceinline__ void rows_load(Run (&r)[4], const RopeParams& rp, const int* pos, const uint16_t* in,
                                          int64_t in_stride, int lane) {
  const Chunks ch = chunks_of<kPairs>(rp, lane);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    load_run(r[u], in + t * in_stride, ch.a, ch.b, pos[t] >= 0);
  }
}
template <bool kPairs>
__device__ __forceinline__ void rows_rotate(const Run (&r)[4], const RopeParams& rp, const float* tab, const int* pos,
                                            uint16_t* out, int64_t out_stride, int lane) {
  const Chunks ch = chunks_of<kPairs>(rp, lane);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    if (pos[t] < 0) continue;
    uint64_t y[8];
    rotate_run<kPairs, false>(r[u], 0, tab + t * kTokStride, lane, ch.rotated, y);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      f2_split(y[i], a, b);
      o[i] = bf16x2_pack(a, b);
    }
    uint16_t* row = out + t * out_stride;
    *reinterpret_cast<uint4*>(row + ch.a) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(row + ch.b) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <bool kPairs>
__device__ __forceinline__ void rows_unit(const RopeParams& rp, const float* tab, const int* pos, const uint16_t* in,
                                          int64_t in_stride, uint16_t* out, int64_t out_stride, int lane) {
  Run r[4];
  rows_load<kPairs>(r, rp, pos, in, in_stride, lane);
  rows_rotate<kPairs>(r, rp, tab, pos, out, out_stride, lane);
}

struct RopeArgs {
  const uint16_t* in[2];       // q, k
  uint16_t* out[2];
  int64_t in_stride[2], out_stride[2];
  int heads[2];                // 0 where absent
  const int32_t* positions;
  int n_tokens;
};

// The rows of a tile's tokens, unit by unit.  fill() forms the table; a warp's first rows are
// on their way meanwhile (8192 tokens of 64 + 8 heads 55.0 -> 51.1 us).  kPairs: rotated pairs
// are neighbouring channels (interleaved style).
template <bool kPairs, class Fill>
__device__ __forceinline__ void rotate_tile(const RopeArgs& a, const RopeParams& rp, const float* tab, const int* pos, int t0,
                                            Fill fill) {
  const int lane = threadIdx.x & 31, units = a.heads[0] + a.heads[1];
  int u = blockIdx.y * kWarps + (threadIdx.x >> 5);
  bool k = u >= a.heads[0];
  Run r[4];
  auto load = [&]() {
    const int64_t is = k ? a.in_stride[1] : a.in_stride[0];
    rows_load<kPairs>(r, rp, pos, (k ? a.in[1] : a.in[0]) + t0 * is + (u - (k ? a.heads[0] : 0)) * 128, is, lane);
  };
  if (u < units) load();
  fill();
  __syncthreads();
  while (u < units) {
    const int64_t os = k ? a.out_stride[1] : a.out_stride[0];
    rows_rotate<kPairs>(r, rp, tab, pos, (k ? a.out[1] : a.out[0]) + t0 * os + (u - (k ? a.heads[0] : 0)) * 128, os, lane);
    u += gridDim.y * kWarps;
    if (u >= units) break;
    k = u >= a.heads[0];
    load();
  }
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(RopeArgs a, const __grid_constant__ RopeParams rp) {
  __shared__ __align__(16) float tab[kTile * kTokStride];
  __shared__ int pos[kTile];
  release_successor();
  after_predecessor();
  const int t0 = blockIdx.x * kTile;
  if (threadIdx.x < kTile) pos[threadIdx.x] = t0 + (int)threadIdx.x < a.n_tokens ? a.positions[t0 + threadIdx.x] : -1;
  __syncthreads();
  rotate_tile<kPairs>(a, rp, tab, pos, t0, [&] { fill_table(tab, rp, pos); });
}

// The same with a position for each axis: a pair turns by that of its own.  Only the
// table differs: 8192 tokens of 64 + 8 heads on three axes 51.1 us by graph replay, 5.9 TB/s,
// 0.88 of a plain copy (one position: 50.5).  64 tokens 4.4 us, 11 with the host's part.
template <bool kPairs>
__global__ void __launch_bounds__(kThreads, 4)
    rope_axes_kernel(RopeArgs a, int64_t pos_stride, const __grid_constant__ RopeAxes axes,
                     const __grid_constant__ RopeParams rp) {
  __shared__ __align__(16) float tab[kTile * kTokStride];
  __shared__ int pos[kTile], at[4][kTile];
  __shared__ __align__(4) uint8_t axis[64];                 // (lanes look at different pairs: not from the parameter)
  release_successor();
  after_predecessor();
  const int t0 = blockIdx.x * kTile;
  if (threadIdx.x >= kTile && threadIdx.x < kTile + 16)
    reinterpret_cast<uint32_t*>(axis)[threadIdx.x - kTile] = reinterpret_cast<const uint32_t*>(axes.axis)[threadIdx.x - kTile];
  if (threadIdx.x < kTile) {
    const int t = threadIdx.x;
    const bool live = t0 + t < a.n_tokens;
    int p[4], low = live ? 0 : -1;             // below 0: a token without work
#pragma unroll
    for (int x = 0; x < 4; ++x) p[x] = live && x < axes.n ? a.positions[x * pos_stride + t0 + t] : low;
#pragma unroll
    for (int x = 0; x < 4; ++x) {              // (no load above waits for another)
      at[x][t] = p[x];
      low = min(low, p[x]);
    }
    pos[t] = low;
  }
  __syncthreads();
  rotate_tile<kPairs>(a, rp, tab, pos, t0, [&] {
    const int n = rp.rd >> 1;
    for (int i = threadIdx.x; i < kTile * 64; i += kThreads) {
      const int t = i >> 6, f = i & 63;
      if (f < n && pos[t] >= 0) {
        const float2 cs = turn_cos_sin((unsigned long long)at[axis[f]][t] * rp.turn[f], rp.att);
        float* d = tab + t * kTokStride + 4 * (f >> 3) + (f & 3) + 32 * ((f >> 2) & 1);
        d[0] = cs.x;
        d[64] = cs.y;
      }
    }
  });
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

// One (tile, head) of K (kV false) or V: tokens [t0, t1) of the tile are new,
// in + t * stride is the row of tile slot t.
template <bool kPairs, bool kV>
__device__ __forceinline__ void quant_unit(const RopeParams& rp, const float* tab, const uint16_t* in, int64_t stride,
                                           int t0, int t1, uint8_t* codes, int8_t* exp, int lane) {
  const Chunks ch = kV ? Chunks{16 * (lane & 7), 16 * (lane & 7) + 8, false} : chunks_of<kPairs>(rp, lane);
  const int e_old = t0 > 0 ? *exp : KV_FP8_EXP_MIN;
  Run r[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    load_run(r[u], in + t * stride, ch.a, ch.b, t >= t0 && t < t1);
  }
  uint32_t bad = 0, mag = 0;                   // passes whose row is not finite; V: the largest magnitude
  float sq = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t m = run_magnitude(r[u]);
    const uint32_t b = __ballot_sync(0xffffffffu, m >= 0x7F80u);
    if ((b >> (lane & 24)) & 0xFFu)
      bad |= 1u << u;
    else if (kV)
      mag = max(mag, m);
    else
      sq = fmaxf(sq, run_square<kPairs>(r[u], rp, ch.rotated));
  }
  // V: a magnitude's exponent by itself (its square would give the same)
  const int e = max(kV ? magnitude_exponent(__reduce_max_sync(0xffffffffu, mag)) : tile_exponent(warp_max_xor(sq, 1)), e_old);
  if (t0 > 0 && e > e_old) {                   // earlier tokens move to the larger exponent
    const float f = pow2i(max(e_old - e, -126));
    for (int t = lane >> 3; t < t0; t += 4) {
      uint4* p = reinterpret_cast<uint4*>(codes + code_offset(kV, t, 16 * (lane & 7)));
      uint4 w = *p;
      w.x = rescale4(w.x, f);
      w.y = rescale4(w.y, f);
      w.z = rescale4(w.z, f);
      w.w = rescale4(w.w, f);
      *p = w;
    }
  }
  const float inv = pow2i(-e);
  const uint64_t inv2 = f2(inv, inv);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 4 * u + (lane >> 3);
    if (t < t0 || t >= t1) continue;
    uint32_t c[4] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
    if (!((bad >> u) & 1)) {
      uint64_t y[8];
      // scaled first: at e = 7 even the largest finite row stays in fp32 while it is rotated
      rotate_run<kPairs, true>(r[u], inv2, tab + t * kTokStride, lane, !kV && ch.rotated, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x0, x1, x2, x3;
        f2_split(y[2 * i], x0, x1);
        f2_split(y[2 * i + 1], x2, x3);
        c[i] = e4m3x4(x0, x1, x2, x3);
      }
    }
    if (kV) {
      *reinterpret_cast<uint4*>(codes + code_offset(true, t, ch.a)) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
      *reinterpret_cast<uint2*>(codes + code_offset(false, t, ch.a)) = make_uint2(c[0], c[1]);
      *reinterpret_cast<uint2*>(codes + code_offset(false, t, ch.b)) = make_uint2(c[2], c[3]);
    }
  }
  if (lane == 0 && (t0 == 0 || e > e_old)) *exp = (int8_t)e;
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) append_fp8_kernel(AppendFp8Args a, const __grid_constant__ RopeParams rp) {
  __shared__ __align__(16) float tab[kTile * kTokStride];
  __shared__ int pos[kTile];
  release_successor();
  after_predecessor();
  const int s = blockIdx.x / a.tiles, i = blockIdx.x - s * a.tiles;
  const int c0 = a.cu[s], c1 = a.cu[s + 1];
  const int start = a.start[s];
  if (c0 < 0 || c1 < c0) {                     // (no difference of these is taken: it could pass 32 bits)
    if (i == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return;
  }
  int n = c1 - c0;
  if (n > a.max_tokens) {
    if (i == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    n = a.max_tokens;
  }
  if (n == 0) return;
  if (start < 0 || (long long)start + n > min((long long)a.max_pages * a.P, (long long)INT32_MAX)) {
    if (i == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return;
  }
  // tile slots [t0, t1) of the i-th tile the sequence's new tokens touch
  const long long base = ((long long)(start / kTile) + i) * kTile;   // position of slot 0
  const long long lo = max(base, (long long)start), hi = min(base + kTile, (long long)start + n);
  if (lo >= hi) return;
  const int t0 = (int)(lo - base), t1 = (int)(hi - base);
  const int lane = threadIdx.x & 31, nkv = 2 * a.Hkv, units = nkv + (a.q ? a.Hq : 0);
  const int first = blockIdx.y * kWarps + (threadIdx.x >> 5);   // this warp's units: first, + gridDim.y * kWarps, ..
  const int64_t row0 = (int64_t)c0 + (base - start);       // input row of slot 0 (rows t0 .. t1 - 1 exist)
  // A unit's rows (half a row per lane) come from memory while the table is formed or
  // the unit before is worked on.
  auto prefetch = [&](int u) {
    const int t = lane >> 1;
    if (u >= units || t < t0 || t >= t1) return;
    const int64_t stride = u < a.Hkv ? a.k_stride : (u < nkv ? a.v_stride : a.q_stride);
    const uint16_t* in = u < a.Hkv ? a.k + u * 128 : (u < nkv ? a.v + (u - a.Hkv) * 128 : a.q + (u - nkv) * 128);
    prefetch_l2(in + (row0 + t) * stride + (lane & 1) * 64);
  };
  prefetch(first);
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
  const int per = a.P / kTile, sub = (int)(base / kTile % per);
  for (int u = first; u < units; u += gridDim.y * kWarps) {
    prefetch(u + gridDim.y * kWarps);
    if (u < nkv) {
      if (!page_ok) continue;
      const int tensor = u >= a.Hkv, h = u - (tensor ? a.Hkv : 0);
      const size_t tile = ((size_t)pid * a.Hkv + h) * per + sub;
      const int64_t stride = tensor ? a.v_stride : a.k_stride;
      uint8_t* codes = a.codes + tile * kFp8TileBytes;
      if (tensor == 0)
        quant_unit<kPairs, false>(rp, tab, a.k + row0 * stride + h * 128, stride, t0, t1, codes, a.exps + tile * 2, lane);
      else
        quant_unit<kPairs, true>(rp, tab, a.v + row0 * stride + h * 128, stride, t0, t1, codes + 2048,
                                 a.exps + tile * 2 + 1, lane);
    } else {
      const int h = u - nkv;
      rows_unit<kPairs>(rp, tab, pos, a.q + row0 * a.q_stride + h * 128, a.q_stride, a.q_out + row0 * a.qo_stride + h * 128,
                a.qo_stride, lane);
    }
  }
}

// Slices of the heads per tile: about `per_sm` CTAs per SM, at most one unit per
// warp.  A slice forms the tile's table again, so the append, whose units are
// longer, takes fewer (8: ragged chunks 55 us, with 4: 61; a prompt of 8192 35,
// with 16: 38) than the rotary rows (16: 51.1 us on three axes, with 8 or 24: 52).
constexpr int kRopePerSm = 16, kAppendPerSm = 8;
unsigned slices(const Pool& p, long long tiles, int units, int per_sm) {
  const long long want = ((long long)per_sm * p.sm_count + tiles - 1) / tiles;
  return (unsigned)std::max(1ll, std::min<long long>((units + kWarps - 1) / kWarps, want));
}

// A speed in radians per position (taken as the double that it is) as turns per position
// modulo one turn, in units of 2^-64, for |w| up to 2^40: 1 / 2 pi in two doubles, the
// product's rounding by fma.
unsigned long long turns_of(double w) {
  constexpr double kInvHi = 0x1.45f306dc9c883p-3, kInvLo = -0x1.6b01ec5417056p-57;
  const double v = std::fabs(w);
  volatile double product = v * kInvHi;          // rounded here, whatever the compiler fuses below
  const double p = product;
  double rest = std::fma(v, kInvHi, -p) + v * kInvLo;
  rest -= std::rint(rest);
  if (rest == 0.5) rest = -0.5;
  const double f = p - std::floor(p), hi = std::floor(std::ldexp(f, 32));
  const double lo = std::ldexp(f, 64) - std::ldexp(hi, 32);
  const unsigned long long t = ((unsigned long long)hi << 32) + (unsigned long long)std::llrint(lo + std::ldexp(rest, 64));
  return w < 0 ? 0ull - t : t;
}

}  // namespace

kv_status_t rope_params(const kv_rope_config_t& c, RopeParams* out) {
  RopeParams r{};
  const int d = c.rotary_dim;
  if (d < 0 || d > 128) return KV_ERR_INVALID_ARG;
  if (d % 32) return KV_ERR_UNSUPPORTED;
  if (c.style != KV_ROPE_HALF && c.style != KV_ROPE_INTERLEAVED) return KV_ERR_INVALID_ARG;
  if (c.scaling < KV_ROPE_SCALE_NONE || c.scaling > KV_ROPE_SCALE_YARN) return KV_ERR_INVALID_ARG;
  // K's exponent goes by its raw rows' squares in fp32 times the factor's, and a row is
  // rotated in units of its tile's scale: within these bounds no square that counts has
  // under- or overflowed, and no finite row passes fp32's range
  if (!(c.attention_factor == 0 || (c.attention_factor >= 1e-12 && c.attention_factor <= 64))) return KV_ERR_INVALID_ARG;
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
      if (att > 64) return KV_ERR_INVALID_ARG;   // as above: a factor beyond e^630
    }
  }
  r.rd = d;
  r.interleaved = c.style == KV_ROPE_INTERLEAVED;
  r.att = (float)(att == 0 ? 1.0 : att);
  r.att2 = (float)((double)r.att * (double)r.att);
  for (int i = 0; i < d / 2; ++i) r.turn[i] = turns_of(w[i]);
  *out = r;
  return KV_OK;
}

namespace {
RopeArgs rope_args(const Pool& p, int n_tokens, const int32_t* positions, const RopeRows& q, const RopeRows& k) {
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
  return a;
}
dim3 rope_grid(const Pool& p, const RopeArgs& a) {
  const long long tiles = ((long long)a.n_tokens + kTile - 1) / kTile;
  return dim3((unsigned)tiles, slices(p, tiles, a.heads[0] + a.heads[1], kRopePerSm));
}
}  // namespace

cudaError_t launch_rope(const Pool& p, const RopeParams& r, int n_tokens, const int32_t* positions, const RopeRows& q,
                        const RopeRows& k, cudaStream_t s) {
  if (n_tokens == 0) return cudaSuccess;
  const RopeArgs a = rope_args(p, n_tokens, positions, q, k);
  return launch_dependent(r.interleaved ? rope_kernel<true> : rope_kernel<false>, rope_grid(p, a), kThreads, 0, s, 1, a, r);
}

cudaError_t launch_rope_axes(const Pool& p, const RopeParams& r, const RopeAxes& x, int n_tokens,
                             const int32_t* positions, int64_t pos_stride, const RopeRows& q, const RopeRows& k,
                             cudaStream_t s) {
  if (n_tokens == 0) return cudaSuccess;
  const RopeArgs a = rope_args(p, n_tokens, positions, q, k);
  return launch_dependent(r.interleaved ? rope_axes_kernel<true> : rope_axes_kernel<false>, rope_grid(p, a), kThreads, 0,
                          s, 1, a, pos_stride, x, r);
}

cudaError_t launch_append_fp8(const Pool& p, const Fp8Store& f, const RopeParams& r, int layer, int n_seqs,
                              const RopeRows& q, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* cu, const int32_t* start, const int32_t* pt, int max_pages,
                              int max_tokens, cudaStream_t s) {
  if (n_seqs == 0) return cudaSuccess;         // (with a bound of 0 a CTA for each sequence still looks at its count)
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
  const dim3 grid((unsigned)tiles, slices(p, tiles, 2 * a.Hkv + (a.q ? a.Hq : 0), kAppendPerSm));
  return launch_dependent(r.interleaved ? append_fp8_kernel<true> : append_fp8_kernel<false>, grid, kThreads, 0, s, 1, a, r);
}

}  // namespace kvint2
