// Writing tokens into the 4-bit cache and reading them back.
//
// Of a block of 16 channels x of a token (as multiples of 2^e, e the layer's exponent):
//   s = e4m3(max |x| / 6),  code = e2m1(x / s),  value = code * s * 2^e.
// Quotients are IEEE ones: the largest magnitude's by division, once per block; x / s by
// the reciprocal r = fl(1 / s) and one correction,  q = q0 + (x - q0 s) r,  q0 = fl(x r),
// in paired fp32 instructions.  What counts is that a quotient halfway between two codes
// comes out exactly, or it would round to the wrong side: q0 misses some of those by a
// last place (s = 15/8 of a power of two times 1.25), q none.  (x of 8 bits over s of 4 is
// otherwise at least 2^-9 away from a halfway point.)
//
// Bound: memory traffic (512 B of rows and 144 B stored per token and KV head) for long
// prompts, latency for single tokens.  A warp owns a (tile, head, tensor): one writer for
// the bytes that two tokens share, no atomics.  A lane quantizes whole blocks (32 bytes
// of a row), so no value crosses lanes: four tokens' blocks each, for V the four tokens
// whose codes share its bytes.
#include <cuda_fp8.h>

#include <algorithm>

#include "kv_device.cuh"
#include "kv_fp4.h"

namespace kvint2 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Four bytes of codes; in each the first value's in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(float a0, float a1, float b0, float b1, float c0, float c1, float d0, float d1) {
  uint32_t r;
  asm("{ .reg .b8 p, q, r, s; cvt.rn.satfinite.e2m1x2.f32 p, %2, %1; cvt.rn.satfinite.e2m1x2.f32 q, %4, %3; "
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5; cvt.rn.satfinite.e2m1x2.f32 s, %8, %7; mov.b32 %0, {p, q, r, s}; }"
      : "=r"(r)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1), "f"(d0), "f"(d1));
  return r;
}

// A block of a row as it comes from memory, and its scale.
struct Block {
  uint32_t w[8];                               // 16 bf16 values
  uint32_t scale;                              // e4m3 byte
  float s, r;                                  // scale * 2^e and its reciprocal
  uint64_t ns2, r2;                            // -s, r as pairs
};

// Read once by this kernel, written perhaps by the one in front, which may have been
// running when this one came up: not the read-only path.
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void load_block(Block& b, const uint16_t* p, bool live) {
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  if (live) {
    x = ld_once(p);
    y = ld_once(p + 8);
  }
  b.w[0] = x.x; b.w[1] = x.y; b.w[2] = x.z; b.w[3] = x.w;
  b.w[4] = y.x; b.w[5] = y.y; b.w[6] = y.z; b.w[7] = y.w;
}

__device__ __forceinline__ void scale_block(Block& b, int e) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, b.w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);               // the largest magnitude's bits
  const float top = bf16lo(m) * pow2i(-e);
  b.scale = m >= 0x7F80u ? 0x7Fu : __nv_cvt_float_to_fp8(__fdiv_rn(top, 6.f), __NV_SATFINITE, __NV_E4M3);
  const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b.scale, __NV_E4M3);
  const float s = __half2float(__half(hr)) * pow2i(e);
  const bool live = m < 0x7F80u && s > 0.f;
  b.s = live ? s : 1.f;
  b.r = live ? __frcp_rn(s) : 0.f;
  if (!live) {                                 // codes of zero
#pragma unroll
    for (int i = 0; i < 8; ++i) b.w[i] = 0;
  } else if (top > 6.f * 448.f) {                     // beyond the format's range: cut where the code is the largest anyway
    const float cut = 7.f * b.s;               // (s = 448 * 2^e: finite)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = fminf(fmaxf(bf16lo(b.w[i]), -cut), cut), y = fminf(fmaxf(bf16hi(b.w[i]), -cut), cut);
      b.w[i] = (__float_as_uint(x) >> 16) | (__float_as_uint(y) & 0xFFFF0000u);   // 7 * 448 * 2^e is a bf16 value
    }
  }
  b.ns2 = f2(-b.s, -b.s);
  b.r2 = f2(b.r, b.r);
}

// The quotients of values 2 i and 2 i + 1.
__device__ __forceinline__ void quotients(const Block& b, int i, float& q0, float& q1) {
  const uint64_t x = f2(bf16lo(b.w[i]), bf16hi(b.w[i])), q = f2_mul(x, b.r2);
  f2_split(f2_fma(f2_fma(q, b.ns2, x), b.r2, q), q0, q1);
}

struct Fp4CacheArgs {
  Fp4Layer L;
  Fp4Tokens t;
  Fp4Rows rows;
  int tiles;                                   // of a sequence, at most
  int* err;
};

// The i-th tile that sequence s's tokens touch: slots [t0, t1) of it, the row of slot 0
// (rows t0 .. t1 - 1 exist), its stored index without the head.  False where there is
// nothing to do.
struct Place {
  int t0, t1, sub;
  long long pid;
  int64_t row0;
};
__device__ __forceinline__ bool find_place(const Fp4CacheArgs& a, int x, Place& p) {
  const int s = x / a.tiles, i = x - s * a.tiles;
  const int c0 = a.t.cu[s], start = a.t.start[s];
  int n = a.t.cu[s + 1] - c0;
  const bool first = i == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  if (n < 0 || n > a.t.max_tokens) {
    if (first) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    n = min(n, a.t.max_tokens);
  }
  if (n <= 0) return false;
  if (start < 0 || (long long)start + n > min((long long)a.t.max_pages * a.L.P, (long long)INT32_MAX)) {
    if (first) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return false;
  }
  const long long base = ((long long)(start / kTile) + i) * kTile;   // position of slot 0
  const long long lo = max(base, (long long)start), hi = min(base + kTile, (long long)start + n);
  if (lo >= hi) return false;
  p.t0 = (int)(lo - base);
  p.t1 = (int)(hi - base);
  p.row0 = (int64_t)c0 + (base - start);
  p.pid = a.t.pt[(size_t)s * a.t.max_pages + base / a.L.P];
  p.sub = (int)(base / kTile % (a.L.P / kTile));
  if (p.pid < 0 || p.pid >= a.L.num_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_PAGE_ID);
    return false;
  }
  return true;
}
__device__ __forceinline__ uint8_t* tile_of(const Fp4CacheArgs& a, const Place& p, int h) {
  return a.L.tiles + ((p.pid * a.L.Hkv + h) * (a.L.P / kTile) + p.sub) * kFp4TileBytes;
}

// K of a tile: lane (t % 4, g) takes block g of tokens t, t + 4, ..
__device__ __forceinline__ void store_k(const uint16_t* in, int64_t stride, int t0, int t1, int e, uint8_t* tile, int lane) {
  const int g = lane & 7, t = lane >> 3;
  Block b[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) load_block(b[u], in + (t + 4 * u) * stride + 16 * g, t + 4 * u >= t0 && t + 4 * u < t1);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (t + 4 * u < t0 || t + 4 * u >= t1) continue;
    scale_block(b[u], e);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float q[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) quotients(b[u], 4 * i + k, q[2 * k], q[2 * k + 1]);
      w[i] = e2m1x8(q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
    }
    *reinterpret_cast<uint2*>(tile + 64 * (t + 4 * u) + 8 * g) = make_uint2(w[0], w[1]);
    tile[kFp4KScale + 8 * (t + 4 * u) + g] = (uint8_t)b[u].scale;
  }
}

// V of a tile: lane (j, g) takes block g of tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9, whose
// codes share its eight words and whose scales its ninth.
__device__ __forceinline__ void store_v(const uint16_t* in, int64_t stride, int t0, int t1, int e, uint8_t* tile, int lane) {
  const int g = lane & 7, j = lane >> 3;
  Block b[4];
  uint32_t mine = 0;                           // bytes of the scale word, halves of the code bytes
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = 2 * j + (u & 1) + 8 * (u >> 1);
    const bool live = t >= t0 && t < t1;
    if (live) mine |= 1u << u;
    load_block(b[u], in + t * stride + 16 * g, live);
  }
  if (mine == 0) return;
  uint32_t scales = 0, byte_mask = 0, code_mask = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    scale_block(b[u], e);
    scales |= b[u].scale << (8 * u);
    if ((mine >> u) & 1) {
      byte_mask |= 0xFFu << (8 * u);
      code_mask |= (u & 1 ? 0xF0F0u : 0x0F0Fu) << (16 * (u >> 1));
    }
  }
  uint32_t* sw = reinterpret_cast<uint32_t*>(tile + kFp4VScale + 32 * j + 4 * g);
  *sw = mine == 15u ? scales : (*sw & ~byte_mask) | (scales & byte_mask);
  uint32_t* cw = reinterpret_cast<uint32_t*>(tile + kFp4V + 512 * (g >> 2) + 16 * j + 4 * (g & 3));   // 16 words apart
  uint32_t old[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) old[i] = mine == 15u ? 0u : cw[16 * i];
#pragma unroll
  for (int i = 0; i < 8; ++i) {                // channels 2 i, 2 i + 1
    float q[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) quotients(b[u], i, q[u][0], q[u][1]);
    const uint32_t w = e2m1x8(q[0][0], q[1][0], q[0][1], q[1][1], q[2][0], q[3][0], q[2][1], q[3][1]);
    cw[16 * i] = (old[i] & ~code_mask) | (w & code_mask);
  }
}

__global__ void __launch_bounds__(kThreads) append_fp4_kernel(Fp4CacheArgs a) {
  release_successor();
  after_predecessor();
  Place p;
  if (!find_place(a, blockIdx.x, p)) return;
  const int lane = threadIdx.x & 31;
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < 2 * a.L.Hkv; u += gridDim.y * kWarps) {
    const int v = u >= a.L.Hkv, h = u - (v ? a.L.Hkv : 0);
    uint8_t* tile = tile_of(a, p, h);
    if (v)
      store_v(static_cast<const uint16_t*>(a.rows.v) + p.row0 * a.rows.v_stride + h * 128, a.rows.v_stride, p.t0, p.t1,
              a.L.v_exp, tile, lane);
    else
      store_k(static_cast<const uint16_t*>(a.rows.k) + p.row0 * a.rows.k_stride + h * 128, a.rows.k_stride, p.t0, p.t1,
              a.L.k_exp, tile, lane);
  }
}

// ---- reading back -----------------------------------------------------------------

__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&f)[4]) {   // fp16 pairs
  asm("{ .reg .b8 p, q, r, s; mov.b32 {p, q, r, s}, %4; cvt.rn.f16x2.e2m1x2 %0, p; cvt.rn.f16x2.e2m1x2 %1, q; "
      "cvt.rn.f16x2.e2m1x2 %2, r; cvt.rn.f16x2.e2m1x2 %3, s; }"
      : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
      : "r"(w));
}
__device__ __forceinline__ float scale_of(uint32_t byte, int e) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(byte & 0xFFu), __NV_E4M3))) * pow2i(e);
}
// two values of one token, times its scale
__device__ __forceinline__ uint32_t bf16_pair(float a, float b, float s) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(a * s, b * s);
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void store_block(uint16_t* p, const uint32_t (&w)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ void load_k(uint16_t* out, int64_t stride, int t0, int t1, int e, const uint8_t* tile, int lane) {
  const int g = lane & 7, t = lane >> 3;
  uint2 w[4];
  uint32_t sc[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    w[u] = *reinterpret_cast<const uint2*>(tile + 64 * (t + 4 * u) + 8 * g);
    sc[u] = tile[kFp4KScale + 8 * (t + 4 * u) + g];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (t + 4 * u < t0 || t + 4 * u >= t1) continue;
    const float s = scale_of(sc[u], e);
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t f[4];
      codes4(i ? w[u].y : w[u].x, f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = __half22float2(u32_as_h2(f[k]));
        y[4 * i + k] = bf16_pair(x.x, x.y, s);
      }
    }
    store_block(out + (t + 4 * u) * stride + 16 * g, y);
  }
}

__device__ __forceinline__ void load_v(uint16_t* out, int64_t stride, int t0, int t1, int e, const uint8_t* tile, int lane) {
  const int g = lane & 7, j = lane >> 3;
  const uint32_t* cw = reinterpret_cast<const uint32_t*>(tile + kFp4V + 512 * (g >> 2) + 16 * j + 4 * (g & 3));
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = cw[16 * i];
  const uint32_t sw = *reinterpret_cast<const uint32_t*>(tile + kFp4VScale + 32 * j + 4 * g);
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {             // tokens 2 j + 8 hi, + 1
    const float s0 = scale_of(sw >> (16 * hi), e), s1 = scale_of(sw >> (16 * hi + 8), e);
    uint32_t y0[8], y1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {              // channels 2 i, 2 i + 1
      uint32_t f[4];
      codes4(w[i], f);
      const float2 a = __half22float2(u32_as_h2(f[2 * hi])), b = __half22float2(u32_as_h2(f[2 * hi + 1]));
      y0[i] = bf16_pair(a.x, b.x, s0);
      y1[i] = bf16_pair(a.y, b.y, s1);
    }
    const int t = 2 * j + 8 * hi;
    if (t >= t0 && t < t1) store_block(out + t * stride + 16 * g, y0);
    if (t + 1 >= t0 && t + 1 < t1) store_block(out + (t + 1) * stride + 16 * g, y1);
  }
}

__global__ void __launch_bounds__(kThreads) read_fp4_kernel(Fp4CacheArgs a) {
  release_successor();
  after_predecessor();
  Place p;
  if (!find_place(a, blockIdx.x, p)) return;
  const int lane = threadIdx.x & 31;
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < 2 * a.L.Hkv; u += gridDim.y * kWarps) {
    const int v = u >= a.L.Hkv, h = u - (v ? a.L.Hkv : 0);
    const uint8_t* tile = tile_of(a, p, h);
    if (v ? a.rows.v == nullptr : a.rows.k == nullptr) continue;
    if (v)
      load_v(static_cast<uint16_t*>(a.rows.v) + p.row0 * a.rows.v_stride + h * 128, a.rows.v_stride, p.t0, p.t1,
             a.L.v_exp, tile, lane);
    else
      load_k(static_cast<uint16_t*>(a.rows.k) + p.row0 * a.rows.k_stride + h * 128, a.rows.k_stride, p.t0, p.t1,
             a.L.k_exp, tile, lane);
  }
}

template <class K>
cudaError_t launch_cache(K kernel, const Pool& p, const Fp4Layer& L, const Fp4Tokens& t, const Fp4Rows& rows, cudaStream_t s) {
  if (t.n_seqs == 0 || t.max_tokens == 0) return cudaSuccess;
  Fp4CacheArgs a{L, t, rows, (int)(((long long)t.max_tokens + 30) / kTile), p.err};   // n tokens touch at most that many tiles
  const dim3 grid((unsigned)((long long)t.n_seqs * a.tiles), (2 * L.Hkv + kWarps - 1) / kWarps);
  return launch_dependent(kernel, grid, kThreads, 0, s, 1, a);
}

}  // namespace

cudaError_t launch_append_fp4(const Pool& p, const Fp4Layer& L, const Fp4Tokens& t, const Fp4Rows& in, cudaStream_t s) {
  return launch_cache(append_fp4_kernel, p, L, t, in, s);
}

cudaError_t launch_read_fp4(const Pool& p, const Fp4Layer& L, const Fp4Tokens& t, const Fp4Rows& out, cudaStream_t s) {
  return launch_cache(read_fp4_kernel, p, L, t, out, s);
}

}  // namespace kvint2
