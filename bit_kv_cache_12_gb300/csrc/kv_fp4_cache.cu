// Writing tokens into the 4-bit cache and reading them back.
//
// Of a block of 16 channels x of a token (as multiples of 2^e, e the layer's exponent):
//   s = e4m3(max |x| / 6),  code = e2m1(x / s),  value = code * s * 2^e.
// The codes are those of exact quotients.  max |x| has 8 bits and its product with
// fl(1 / 6) comes out exactly where the quotient lies halfway between two e4m3 numbers (the
// constant is off by 2^-25 of itself, less than half a last place of any such number), and on the
// right side of it elsewhere.  x / s is the product with a reciprocal that is off by a last
// place or two of fp32, rounded to fp16 on the way to e2m1: a quotient halfway between two
// codes (3 bits) comes out exactly, and as x of 8 bits over s of 4 is otherwise at least 2^-9
// away from a halfway point, no other quotient (2^-11 off) reaches one.
//
// Bound: memory traffic (512 B of rows and 144 B stored per token and KV head) for long
// prompts, latency for single tokens.  A warp owns a (tile, head, tensor): one writer for
// the bytes that two tokens share, no atomics.  16 lanes take a token's row, 16 bytes each,
// so every load and store of rows is of whole lines (with eight lanes and 32 bytes each an
// append of 8192 tokens took 15.0 us, reading 8 x 6500 back 57.8); two lanes share a block
// and exchange its maximum.
//
// Measured (8 KV heads): append of 8192 tokens 10.2 us, 8.3 to read them back, of which 2.5
// are the launch and rows and tiles fit in the L2 cache; ragged appends and reads of 8 x 6500
// tokens on average 51.9 and 44.7 us (273 MB: 5.3 and 6.1 TB/s, 0.79 and 0.91 of a plain
// copy), with 60% of the issue slots in use; a token of each of 64 sequences 3.6 us, a
// 1000-token prefix back 3.2 (launch and latency).  CTAs of 128 threads, a tile and up to two
// heads each: with 256 the ragged append took 57.6 us.  Seven of them per SM for the append
// (72 registers; with eight 10.6 us and 3.9), eight for the read.
#include <cuda_fp8.h>

#include <algorithm>

#include "kv_device.cuh"
#include "kv_fp4.h"

namespace kvint2 {

namespace {

constexpr int kThreads = 128;
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
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Four bytes of codes from four fp16 pairs; in each the first value's in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  uint32_t r;
  asm("{ .reg .b8 p, q, r, s; cvt.rn.satfinite.e2m1x2.f16x2 p, %1; cvt.rn.satfinite.e2m1x2.f16x2 q, %2; "
      "cvt.rn.satfinite.e2m1x2.f16x2 r, %3; cvt.rn.satfinite.e2m1x2.f16x2 s, %4; mov.b32 %0, {p, q, r, s}; }"
      : "=r"(r)
      : "r"(a), "r"(b), "r"(c), "r"(d));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }

// Read once by this kernel, written perhaps by the one in front, which may have been
// running when this one came up: not the read-only path.
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {   // of bf16 pairs; NaN wins
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Half a block, eight channels of a token; this lane's neighbour (lane ^ 1) has the other.
struct Half {
  uint32_t w[4];                               // bf16 pairs
  uint32_t scale;                              // the block's, e4m3
  uint64_t r2;                                 // 1 / (s * 2^e), twice
};

// Of a block the largest magnitude's bits, from what both lanes hold (above 0x7F7F: not all
// are finite).
__device__ __forceinline__ uint32_t magnitude(const Half& b) {
  uint32_t m = larger(larger(b.w[0] & 0x7FFF7FFFu, b.w[1] & 0x7FFF7FFFu), larger(b.w[2] & 0x7FFF7FFFu, b.w[3] & 0x7FFF7FFFu));
  m = larger(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return larger(m, m >> 16) & 0xFFFFu;
}

// A block whose codes do not come by the usual way: zeros, or cut where they are the largest anyway.
__device__ __forceinline__ void unusual(Half& b, uint32_t m, float& s) {
  if (m >= 0x7F80u || s == 0.f) {
    if (m >= 0x7F80u) b.scale = 0x7Fu;
    s = 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = 0;
  } else {
    const float cut = 7.f * s;                 // (finite, and a bf16 value)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = fminf(fmaxf(bf16lo(b.w[i]), -cut), cut), y = fminf(fmaxf(bf16hi(b.w[i]), -cut), cut);
      b.w[i] = (__float_as_uint(x) >> 16) | (__float_as_uint(y) & 0xFFFF0000u);
    }
  }
}

// The scales of two blocks.  sixth: fl(1 / 6) * 2^-e, unit: 2^e.
__device__ __forceinline__ void scale_blocks(Half& a, Half& b, float sixth, float unit) {
  const uint32_t ma = magnitude(a), mb = magnitude(b);
  const float ta = bf16lo(ma) * sixth, tb = bf16lo(mb) * sixth;
  uint32_t pair, half;
  asm("{ .reg .b16 p; cvt.rn.satfinite.e4m3x2.f32 p, %2, %3; cvt.u32.u16 %0, p; cvt.rn.f16x2.e4m3x2 %1, p; }"
      : "=r"(pair), "=r"(half)
      : "f"(tb), "f"(ta));
  const float2 s2 = __half22float2(u32_as_h2(half));
  float sa = s2.x * unit, sb = s2.y * unit, ra, rb;
  a.scale = pair & 0xFFu;
  b.scale = pair >> 8;
  // beyond the range (tops of 2688 and more, not finite ones among them), or all zeros
  if (__any_sync(0xffffffffu, !(fmaxf(ta, tb) < 448.f) || fminf(sa, sb) == 0.f || max(ma, mb) >= 0x7F80u)) {
    if (!(ta < 448.f) || sa == 0.f || ma >= 0x7F80u) unusual(a, ma, sa);
    if (!(tb < 448.f) || sb == 0.f || mb >= 0x7F80u) unusual(b, mb, sb);
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ra) : "f"(sa));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rb) : "f"(sb));
  a.r2 = f2(ra, ra);
  b.r2 = f2(rb, rb);
}

// The quotients of values 2 i and 2 i + 1.
__device__ __forceinline__ void quotients(const Half& b, int i, float& q0, float& q1) {
  f2_split(f2_mul(f2(bf16lo(b.w[i]), bf16hi(b.w[i])), b.r2), q0, q1);
}

struct Fp4CacheArgs {
  Fp4Layer L;
  Fp4Tokens t;
  Fp4Rows rows;
  int tiles;                                   // of a sequence, at most
  int* err;
};

// The i-th tile that sequence s's tokens touch: slots [t0, t1) of it, the row of slot 0
// (rows t0 .. t1 - 1 exist), its page, as the table has it, and its place there.  False where
// there is nothing to do.
struct Place {
  int t0, t1, pid, sub;
  int64_t row0;
};
__device__ __forceinline__ bool find_place(const Fp4CacheArgs& a, int x, Place& p) {
  const int s = x / a.tiles, i = x - s * a.tiles;
  const int c0 = a.t.cu[s], c1 = a.t.cu[s + 1], start = a.t.start[s];
  const bool first = i == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  if (c0 < 0 || c1 < c0) {                     // (no difference of these is taken: it could pass 32 bits)
    if (first) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return false;
  }
  int n = c1 - c0;
  if (n > a.t.max_tokens) {
    if (first) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    n = a.t.max_tokens;
  }
  if (n == 0) return false;
  if (start < 0 || (long long)start + n > min((long long)a.t.max_pages * a.L.P, (long long)INT32_MAX)) {
    if (first) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return false;
  }
  // a position is below 2^31: so is that of slot 0 of its tile, and tiles behind the last are not touched
  const int tile = start / kTile + i;
  if (tile > (start + n - 1) / kTile) return false;
  const int base = tile * kTile;
  p.t0 = max(start - base, 0);
  p.t1 = min(start + n - base, kTile);
  p.row0 = (int64_t)c0 + base - start;
  p.pid = a.t.pt[(size_t)s * a.t.max_pages + base / a.L.P];
  p.sub = tile & (a.L.P / kTile - 1);
  return true;
}
__device__ __forceinline__ bool good_page(const Fp4CacheArgs& a, const Place& p) {
  if (p.pid >= 0 && p.pid < a.L.num_pages) return true;
  if (blockIdx.y == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_PAGE_ID);
  return false;
}
__device__ __forceinline__ uint8_t* tile_of(const Fp4CacheArgs& a, const Place& p, int h) {
  return a.L.tiles + (((size_t)p.pid * a.L.Hkv + h) * (a.L.P / kTile) + p.sub) * kFp4TileBytes;
}

// The slot of a tile whose row a lane's u-th load or store of K, of V is of.
__device__ __forceinline__ int k_slot(int u, int lane) { return 2 * u + (lane >> 4); }
__device__ __forceinline__ int v_slot(int u, int lane) { return 4 * (u >> 2) + 2 * (lane >> 4) + (u & 1) + 8 * ((u >> 1) & 1); }

// K of a tile; x: this lane's eight pieces of rows.
__device__ __forceinline__ void store_k(const uint4 (&x)[8], int t0, int t1, int e, uint8_t* tile, int lane) {
  const int c = lane & 15;
  const float sixth = 0x1.555556p-3f * pow2i(-e), unit = pow2i(e);
#pragma unroll
  for (int u = 0; u < 8; u += 2) {
    Half b[2] = {{{x[u].x, x[u].y, x[u].z, x[u].w}}, {{x[u + 1].x, x[u + 1].y, x[u + 1].z, x[u + 1].w}}};
    scale_blocks(b[0], b[1], sixth, unit);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float q0, q1;
        quotients(b[v], i, q0, q1);
        q[i] = pack_f16(q0, q1);
      }
      const uint32_t w = e2m1x8(q[0], q[1], q[2], q[3]);
      const int t = k_slot(u + v, lane);
      if (t >= t0 && t < t1) {
        *reinterpret_cast<uint32_t*>(tile + 64 * t + 4 * c) = w;
        if ((c & 1) == 0) tile[kFp4KScale + 8 * t + (c >> 1)] = (uint8_t)b[v].scale;
      }
    }
  }
}

// V of a tile.  Four loads are of the tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9, whose codes share
// the lane's four words and whose scales share one.
__device__ __forceinline__ void store_v(const uint4 (&x)[8], int t0, int t1, int e, uint8_t* tile, int lane) {
  const int c = lane & 15, g = c >> 1;
  const float sixth = 0x1.555556p-3f * pow2i(-e), unit = pow2i(e);
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int j = 2 * v + (lane >> 4);
    Half b[4];
    uint32_t scales = 0, byte_mask = 0, code_mask = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4& y = x[4 * v + u];
      b[u].w[0] = y.x, b[u].w[1] = y.y, b[u].w[2] = y.z, b[u].w[3] = y.w;
      if (u & 1) scale_blocks(b[u - 1], b[u], sixth, unit);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      scales |= b[u].scale << (8 * u);
      const int t = v_slot(4 * v + u, lane);
      if (t >= t0 && t < t1) {
        byte_mask |= 0xFFu << (8 * u);
        code_mask |= (u & 1 ? 0xF0F0u : 0x0F0Fu) << (16 * (u >> 1));
      }
    }
    uint32_t* sw = reinterpret_cast<uint32_t*>(tile + kFp4VScale + 32 * j + 4 * g);
    uint32_t* cw = reinterpret_cast<uint32_t*>(tile + kFp4V + 512 * (g >> 2) + 256 * (c & 1) + 16 * j + 4 * (g & 3));
    uint32_t old[4] = {}, os = 0;              // cw: 16 words apart
    if (byte_mask != 0 && byte_mask != 0xFFFFFFFFu) {
      os = *sw;
#pragma unroll
      for (int i = 0; i < 4; ++i) old[i] = cw[16 * i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float q[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) quotients(b[u], i, q[u][0], q[u][1]);
      const uint32_t w = e2m1x8(pack_f16(q[0][0], q[1][0]), pack_f16(q[0][1], q[1][1]), pack_f16(q[2][0], q[3][0]),
                                pack_f16(q[2][1], q[3][1]));
      if (byte_mask) cw[16 * i] = (old[i] & ~code_mask) | (w & code_mask);
    }
    if (byte_mask && (c & 1) == 0) *sw = (os & ~byte_mask) | (scales & byte_mask);
  }
}

__global__ void __launch_bounds__(kThreads, 7) append_fp4_kernel(Fp4CacheArgs a) {
  release_successor();
  after_predecessor();
  Place p;
  if (!find_place(a, blockIdx.x, p)) return;
  const int lane = threadIdx.x & 31;
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < 2 * a.L.Hkv; u += gridDim.y * kWarps) {
    const bool v = u >= a.L.Hkv;
    const int h = u - (v ? a.L.Hkv : 0);
    const int64_t stride = v ? a.rows.v_stride : a.rows.k_stride;
    const uint16_t* in = static_cast<const uint16_t*>(v ? a.rows.v : a.rows.k) + p.row0 * stride + h * 128 + 8 * (lane & 15);
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = v ? v_slot(i, lane) : k_slot(i, lane);
      x[i] = make_uint4(0, 0, 0, 0);
      if (t >= p.t0 && t < p.t1) x[i] = ld_once(in + t * stride);
    }
    if (!good_page(a, p)) return;              // (its id came with the rows)
    uint8_t* tile = tile_of(a, p, h);
    if (v)
      store_v(x, p.t0, p.t1, a.L.v_exp, tile, lane);
    else
      store_k(x, p.t0, p.t1, a.L.k_exp, tile, lane);
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

// First to leave the L2 cache, so that the tiles stay: 8192 tokens of three layers in turn 10.1
// -> 8.3 us; prompt attention over the rows behind it takes the same (78.1 and 78.1 us for 512
// queries, 41.7 and 42.2 for 64).
__device__ __forceinline__ void put_row(uint16_t* to, const uint32_t (&y)[4]) {
  __stcs(reinterpret_cast<uint4*>(to), make_uint4(y[0], y[1], y[2], y[3]));
}

__device__ __forceinline__ void load_k(uint16_t* out, int64_t stride, int t0, int t1, int e, const uint8_t* tile, int lane) {
  const int c = lane & 15;
  uint32_t w[8], sc[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int t = k_slot(u, lane);
    w[u] = *reinterpret_cast<const uint32_t*>(tile + 64 * t + 4 * c);
    sc[u] = tile[kFp4KScale + 8 * t + (c >> 1)];
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int t = k_slot(u, lane);
    if (t < t0 || t >= t1) continue;
    const float s = scale_of(sc[u], e);
    uint32_t f[4];
    codes4(w[u], f);
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = __half22float2(u32_as_h2(f[k]));
      y[k] = bf16_pair(x.x, x.y, s);
    }
    put_row(out + t * stride + 8 * c, y);
  }
}

__device__ __forceinline__ void load_v(uint16_t* out, int64_t stride, int t0, int t1, int e, const uint8_t* tile, int lane) {
  const int c = lane & 15, g = c >> 1;
  uint32_t w[2][4], sw[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int j = 2 * v + (lane >> 4);
    const uint32_t* cw = reinterpret_cast<const uint32_t*>(tile + kFp4V + 512 * (g >> 2) + 256 * (c & 1) + 16 * j + 4 * (g & 3));
#pragma unroll
    for (int i = 0; i < 4; ++i) w[v][i] = cw[16 * i];
    sw[v] = *reinterpret_cast<const uint32_t*>(tile + kFp4VScale + 32 * j + 4 * g);
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint32_t f[4][4];                          // [channels 2 i, 2 i + 1 of two][two tokens of four]
#pragma unroll
    for (int i = 0; i < 4; ++i) codes4(w[v][i], f[i]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = v_slot(4 * v + u, lane);
      if (t < t0 || t >= t1) continue;
      const float s = scale_of(sw[v] >> (8 * u), e);
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = __half22float2(u32_as_h2(f[i][2 * (u >> 1)])), b = __half22float2(u32_as_h2(f[i][2 * (u >> 1) + 1]));
        y[i] = u & 1 ? bf16_pair(a.y, b.y, s) : bf16_pair(a.x, b.x, s);
      }
      put_row(out + t * stride + 8 * c, y);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 8) read_fp4_kernel(Fp4CacheArgs a) {
  release_successor();
  after_predecessor();
  Place p;
  if (!find_place(a, blockIdx.x, p) || !good_page(a, p)) return;
  const int lane = threadIdx.x & 31;
  for (int u = blockIdx.y * kWarps + (threadIdx.x >> 5); u < 2 * a.L.Hkv; u += gridDim.y * kWarps) {
    const bool v = u >= a.L.Hkv;
    const int h = u - (v ? a.L.Hkv : 0);
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
  if (t.n_seqs == 0) return cudaSuccess;       // (with a bound of 0 a CTA for each sequence still looks at its count)
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
