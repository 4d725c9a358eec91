// Single-token attention over the 8-bit cache, split over the cache.
//
// With code values k, v (e4m3) of tile exponents eK, eV and base-2 logits
//   x_j = scale log2(e) (q . k_j) 2^eK + eV,   w_j = 2^(x_j - M),
// a head's output is  sum_j w_j v_j / sum_j w_j 2^-eV : the V scale rides on the
// weight, so the products use the codes as they are, and the reference M follows
// the largest weight times V scale.  -64 <= eV <= 7 keeps every sum in fp32.
//
// Both products are m16n8k16 tensor-core steps with the cached tile as the A
// operand and the (up to 8) query heads of the KV head as the 8 columns: e4m3
// converts to fp16 exactly (one instruction for two codes).  q enters as fp16
// scaled per head by a power of two (its largest element in [2^14, 2^15)):
// exact for all of bf16's 8 bits down to 2^-32 of the largest, 2^-39 of it
// beyond, below the rounding of the fp32 sum.  The weights are rounded to fp16
// (11 bits) relative to their own size; M lags so that they stay between 2^-31
// of the largest and 2^15.
//
// Bound: HBM (256 B and 2 exponent bytes per token and KV head).  Each warp
// streams whole 4 KB tiles through a ring of its own (bulk copies, no block
// barrier in the loop); the stored order is the operand order, so every lane
// reads its fragments as 16-byte pieces without bank conflicts.  The work of a
// (sequence, KV head) is split over CTAs by the sequence's own count of visible
// tiles.  Up to eight splits of a pair, all on the device at once, are a cluster and
// read one another's parts from shared memory (1024 tokens 4.8 us, of which 3.0 are an
// empty call's; 6.7 through global memory); else the last CTA to finish joins the
// parts.  Both go in split order: the result does not depend on timing.
// 100,000 tokens (32 query heads, 8 KV heads): 39.1 us, 5.2 TB/s, 0.78 of a plain
// copy's rate (4 us to the first tile, 4 for the join, 1.4 since large logits are
// kept in range); 64 sequences of 8k to 32k tokens: 399 us, 6.9 TB/s, 1.03 of it (a
// copy also writes).
#include <algorithm>
#include <atomic>

#include "kv_device.cuh"
#include "kv_fp8.h"

namespace kvint2 {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;                     // 4 KB tiles in flight per warp
constexpr int kPolls = 1 << 18;                // bound of a copy's wait: a poll suspends for up to 3.7 us, so about a second
constexpr int kMaxSplits = 64;
constexpr int kMaxCluster = 8;                 // the portable cluster size
constexpr int kPart = 132;                     // floats of a partial head: M, l, 2 unused, 128 sums
constexpr float kNoRef = -3e38f;               // below every logit
constexpr float kRaise = 15.f, kHead = 7.f;    // M moves when x > M + 15, to the largest x - 7
constexpr uint32_t kRing = kWarps * kStages * kFp8TileBytes;
constexpr uint32_t kSmem = kRing + kWarps * kStages * 8;
// results of the warps in shared memory (over the ring): channel c of a head at
// c + 4 (c / 16), heads 161 floats apart: few bank conflicts for either side
constexpr int kHeadStride = 161;
__device__ __forceinline__ int chan(int c) { return c + 4 * (c >> 4); }

struct DecodeFp8Args {
  Fp8Layer L;
  AttnCall c;
  int B, Hq, n_split;
  unsigned* tickets;
  int* err;
  int polls;
  int stall;                                   // test hook: warp 0 of CTA 0 never starts its first copy
  int cluster;                                 // the splits of a pair are a cluster
};

// The tiles a query at position n - 1 sees: the first `ns`, then those from
// w0 on.
struct Span {
  int n, low, sinks, ns, w0, total;
  __device__ __forceinline__ Span(int len, int window, int n_sink) {
    n = len;
    low = window ? max(len - window, 0) : 0;
    sinks = window ? min(n_sink, len) : 0;
    w0 = low / kTile;
    ns = min((sinks + kTile - 1) / kTile, w0);
    total = ns + (len + kTile - 1) / kTile - w0;
  }
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : i - ns + w0; }
  // bit t: token t of the tile is visible
  __device__ __forceinline__ uint32_t mask(int tile) const {
    const int t0 = tile * kTile;
    auto below = [&](int j) { return j <= t0 ? 0u : (j - t0 >= kTile ? 0xFFFFu : (1u << (j - t0)) - 1u); };
    return below(n) & (~below(low) | below(sinks));
  }
};

__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) {   // codes in bytes 0, 1 -> fp16x2
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) {   // bytes 2, 3
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// p of the cluster's CTA `rank`
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_remote2(uint32_t p) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_remote4(uint32_t p) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(p)
               : "memory");
  return v;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 2) decode_fp8_kernel(DecodeFp8Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  uint8_t* ring = smem + warp * kStages * kFp8TileBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kRing) + warp * kStages;
  if (lane < kStages) mbar_init(bar + lane, 1);
  mbar_fence_init();
  __syncwarp();
  release_successor();
  after_predecessor();

  const int split = blockIdx.x % a.n_split, pair = blockIdx.x / a.n_split;
  const int h = pair % a.L.Hkv, b = pair / a.L.Hkv;
  int n = a.c.seq_len[b];
  // lane (r, j) holds head r, channels 64 c + 16 j + 0..15; on its way with the length
  uint32_t qf[2][8];
  {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.c.q) +
                                                    ((size_t)b * a.Hq + h * G + (r < G ? r : 0)) * 128);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 x = q[8 * c + 2 * j], y = q[8 * c + 2 * j + 1];
      const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) qf[c][i] = w[i];
    }
  }
  if (n < 0 || n > a.c.max_len) {
    if (split == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_LENGTH);
    n = min(max(n, 0), a.c.max_len);
  }
  const Span sp(n, a.c.window, a.c.n_sink);
  const int per = (sp.total + a.n_split - 1) / a.n_split;
  const int i0 = split * per, count = max(min(per, sp.total - i0), 0);
  const int mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;   // tiles i0 + warp, + kWarps, ..
  const int tpp = a.L.P / kTile, tpp_shift = tpp >> 1;
  const int32_t* pt = a.c.pt + (size_t)b * a.c.max_pages;

  // The warp's k-th tile: its page id is read a batch of 32 tiles ahead and not
  // looked at before its turn (no load below waits for another where it is issued).
  auto page_of = [&](int k) -> int {
    return pt[k < mine ? sp.tile(i0 + warp + k * kWarps) >> tpp_shift : 0];
  };
  auto stored = [&](int k, int pid) -> long long {   // -1: no such tile, or behind a bad page id
    if (k >= mine) return -1;
    if (pid < 0 || pid >= a.L.num_pages) {
      flag_error(a.err, KV_DEVERR_PAGE_ID);
      return -1;
    }
    return ((long long)pid * a.L.Hkv + h) * tpp + (sp.tile(i0 + warp + k * kWarps) & (tpp - 1));
  };
  auto exps_of = [&](long long t) -> int {
    return *reinterpret_cast<const uint16_t*>(a.L.exps + max(t, 0ll) * 2);
  };
  const uint64_t policy = l2_evict_first_policy();
  auto issue = [&](int stage, long long t) {     // lane 0
    if (t < 0) {
      mbar_expect_tx(bar + stage, 0);
    } else {
      mbar_expect_tx(bar + stage, kFp8TileBytes);
      bulk_g2s_hint(ring + stage * kFp8TileBytes, a.L.codes + t * kFp8TileBytes, kFp8TileBytes, bar + stage, policy);
    }
  };
  // lane l knows the l-th tile of the current 32 and the page id of the next
  const int pid0 = page_of(lane);
  int next_pid = page_of(32 + lane);
  long long cur = stored(lane, pid0), next = -1;
#pragma unroll
  for (int k = 0; k < kStages; ++k) {
    const long long t = __shfl_sync(0xffffffffu, cur, k);
    if (lane != 0 || k >= mine) continue;
    if (a.stall && k == 0 && blockIdx.x == 0 && warp == 0)
      mbar_expect_tx(bar, kFp8TileBytes);
    else
      issue(k, t);
  }
  int exps = exps_of(cur);

  // q as the B operand: scaled per head by a power of two, fp16
  float cs0, cs1;
  {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (r >= G) qf[i >> 3][i & 7] = 0;       // columns without a head
      const uint32_t w = qf[i >> 3][i & 7];
      top = max(top, max(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int up = min(14 - ((int)(top >> 7) - 127), 127);
    const float mul = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : pow2i(up);   // not finite: NaN
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t w = qf[i >> 3][i & 7];
      qf[i >> 3][i & 7] = pack_f16(bf16lo(w) * mul, bf16hi(w) * mul);
    }
    const float cs = a.c.scale * 1.4426950408889634f * pow2i(max(-up, -126));
    cs0 = __shfl_sync(0xffffffffu, cs, 8 * j);          // heads 2j, 2j + 1
    cs1 = __shfl_sync(0xffffffffu, cs, 8 * j + 4);
  }

  float M0 = kNoRef, M1 = kNoRef, l0 = 0.f, l1 = 0.f;
  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  bool ok = true, large = false;               // large: some head's reference is
  int k = 0, stage = 0, phase = 0;
  for (; k < mine; ++k) {
    if ((k & 31) == 0) {                       // the next 32: their page ids have been on the way since the last batch
      if (k) {
        cur = next;
        exps = exps_of(cur);
      }
      next = stored(k + 32 + lane, next_pid);
      next_pid = page_of(k + 64 + lane);
    }
    // the lanes vote: a copy that lands just as the limit runs out must not part them
    if (!__all_sync(0xffffffffu, mbar_wait(bar + stage, phase, a.polls))) {
      ok = false;
      break;
    }
    const int e2 = __shfl_sync(0xffffffffu, exps, k & 31);
    const bool have = __shfl_sync(0xffffffffu, (int)(cur >= 0), k & 31);
    if (have) {
      const int tile = sp.tile(i0 + warp + k * kWarps);
      const uint32_t vis = sp.mask(tile);
      const uint8_t* codes = ring + stage * kFp8TileBytes + lane * 16;
      uint4 kw[4], vw[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) kw[p] = *reinterpret_cast<const uint4*>(codes + p * 512);
#pragma unroll
      for (int p = 0; p < 4; ++p) vw[p] = *reinterpret_cast<const uint4*>(codes + 2048 + p * 512);
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = (&kw[0].x)[w], a1 = (&kw[2].x)[w], b0 = (&kw[1].x)[w], b1 = (&kw[3].x)[w];
        mma_f16(sa, cvt_lo(a0), cvt_lo(a1), cvt_hi(a0), cvt_hi(a1), qf[0][2 * w], qf[0][2 * w + 1]);
        mma_f16(sb, cvt_lo(b0), cvt_lo(b1), cvt_hi(b0), cvt_hi(b1), qf[1][2 * w], qf[1][2 * w + 1]);
      }
      const float ev = (float)(int8_t)(e2 >> 8), fk = exp2f((float)(int8_t)(e2 & 0xFF));
      float c0 = cs0 * fk, c1 = cs1 * fk;
      float s0 = sa[0] + sb[0], s1 = sa[1] + sb[1];      // token r, heads 2j, 2j + 1
      float s2 = sa[2] + sb[2], s3 = sa[3] + sb[3];      // token r + 8
      float x0 = fmaf(s0, c0, ev), x1 = fmaf(s1, c1, ev), x2 = fmaf(s2, c0, ev), x3 = fmaf(s3, c1, ev);
      if (vis != 0xFFFFu) {                    // hidden tokens: no weight, and codes of zero
        if (!((vis >> r) & 1)) x0 = x1 = -INFINITY;
        if (!((vis >> (r + 8)) & 1)) x2 = x3 = -INFINITY;
        const uint32_t v4 = (vis >> (2 * j)) & 3u, v5 = (vis >> (2 * j + 8)) & 3u;
        const uint4 z = make_uint4(0, 0, 0, 0);
        if (!(v4 & 1)) vw[0] = z;
        if (!(v4 & 2)) vw[1] = z;
        if (!(v5 & 1)) vw[2] = z;
        if (!(v5 & 2)) vw[3] = z;
      }
      float d0 = ev - M0, d1 = ev - M1;
      if (__any_sync(0xffffffffu, large || fmaxf(x0, x2) > M0 + kRaise || fmaxf(x1, x3) > M1 + kRaise)) {
        // as differences: where M is large, M + 15 is rounded by as much as that
        const float t0 = warp_max_xor(fmaxf(x0, x2), 4), t1 = warp_max_xor(fmaxf(x1, x3), 4);
        const float n0 = t0 - M0 > kRaise ? t0 - kHead : M0, n1 = t1 - M1 > kRaise ? t1 - kHead : M1;
        const float f0 = exp2_neg(M0 - n0), f1 = exp2_neg(M1 - n1);
        M0 = n0;
        M1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f1;
          o[i][2] *= f0;
          o[i][3] *= f1;
        }
        d0 = ev - M0;
        d1 = ev - M1;
        const bool g0 = large_reference(M0), g1 = large_reference(M1);
        large = __any_sync(0xffffffffu, g0 || g1);
        // weights from the rounded logits; in here, so that the usual tile has no more to
        // do (100,000 tokens: 39.0 us; with a choice at each weight 39.4 to 40.2)
        if (g0) s0 = x0 - M0, s2 = x2 - M0, c0 = 1.f, d0 = 0.f;
        if (g1) s1 = x1 - M1, s3 = x3 - M1, c1 = 1.f, d1 = 0.f;
      }
      // once more against M: x was rounded at eV's size, ev - M is exact near the largest weight
      auto weight = [](float x, float y) { return x == -INFINITY ? 0.f : exp2_neg(y); };   // -inf: hidden
      const float w0 = weight(x0, fmaf(s0, c0, d0)), w1 = weight(x1, fmaf(s1, c1, d1));
      const float w2 = weight(x2, fmaf(s2, c0, d0)), w3 = weight(x3, fmaf(s3, c1, d1));
      const float fv = exp2f(-ev);
      l0 = fmaf(w0 + w2, fv, l0);
      l1 = fmaf(w1 + w3, fv, l1);
      const uint32_t p0 = movmatrix_t(pack_f16(w0, w1)), p1 = movmatrix_t(pack_f16(w2, w3));
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t v0 = (&vw[0].x)[w], v1 = (&vw[1].x)[w], v2 = (&vw[2].x)[w], v3 = (&vw[3].x)[w];
        const uint32_t a = __byte_perm(v0, v1, 0x5140), bb = __byte_perm(v2, v3, 0x5140);
        const uint32_t c = __byte_perm(v0, v1, 0x7362), d = __byte_perm(v2, v3, 0x7362);
        mma_f16(o[2 * w], cvt_lo(a), cvt_hi(a), cvt_lo(bb), cvt_hi(bb), p0, p1);       // channels 16 r + 4 w + 0, 1
        mma_f16(o[2 * w + 1], cvt_lo(c), cvt_hi(c), cvt_lo(d), cvt_hi(d), p0, p1);     // + 2, 3
      }
    }
    __syncwarp();
    const int kn = k + kStages;
    if (kn < mine) {
      const long long t = __shfl_sync(0xffffffffu, (kn >> 5) == (k >> 5) ? cur : next, kn & 31);
      if (lane == 0) issue(stage, t);
    }
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!ok) {
    // A copy did not arrive in time.  Those in flight, this one among them, would land on
    // what is written over the ring: they are waited for, by the full limit (but not for
    // one that the test hook never started).
    if (lane == 0) flag_error(a.err, KV_DEVERR_TIMEOUT);
    for (int kk = k; kk < min(mine, k + kStages); ++kk) {
      if (!(a.stall && kk == 0 && blockIdx.x == 0 && warp == 0)) mbar_wait(bar + stage, phase, kPolls);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    __syncwarp();
    M0 = M1 = kNoRef;
    l0 = l1 = 0.f;
  }

  // ---- the warps' results -> the CTA's ----
  __syncthreads();                             // every warp is done with its ring
  float* wo = reinterpret_cast<float*>(smem);
  float* wm = wo + kWarps * G * kHeadStride;   // [warp][head] M, then l
  float* wl = wm + kWarps * G;
  l0 = warp_sum_xor(l0, 4);
  l1 = warp_sum_xor(l1, 4);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int g = 2 * j + u;
    if (g < G) {
      float* d = wo + (warp * G + g) * kHeadStride;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[chan(16 * r + 2 * i)] = o[i][u];
        d[chan(16 * r + 2 * i + 1)] = o[i][2 + u];
      }
      if (r == 0) {
        wm[warp * G + g] = u ? M1 : M0;
        wl[warp * G + g] = u ? l1 : l0;
      }
    }
  }
  __syncthreads();
  uint16_t* out = static_cast<uint16_t*>(a.c.out) + ((size_t)b * a.Hq + h * G) * 128;
  float* lse = a.c.lse ? a.c.lse + (size_t)b * a.Hq + h * G : nullptr;
  float* parts = static_cast<float*>(a.c.ws) + (size_t)pair * a.n_split * G * kPart;
  float* own = wl + ((kWarps * G + 3) & ~3);   // cluster: this split's part
  for (int idx = threadIdx.x; idx < G * 128; idx += kThreads) {
    const int g = idx >> 7, c = idx & 127;
    float M = kNoRef;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * G + g]);
    float l = 0.f, s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = wl[w * G + g] == 0.f ? 0.f : exp2_neg(wm[w * G + g] - M);
      l = fmaf(f, wl[w * G + g], l);
      if (wl[w * G + g] != 0.f) s = fmaf(f, wo[(w * G + g) * kHeadStride + chan(c)], s);
    }
    if (a.n_split == 1) {
      const float y = l == 0.f ? 0.f : s / l;
      out[g * 128 + c] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      if (c == 0 && lse) lse[g] = lse_of(M, l);
    } else {
      float* p = a.cluster ? own + g * kPart : parts + ((size_t)split * G + g) * kPart;
      p[4 + c] = s;
      if (c == 0) {
        p[0] = M;
        p[1] = l;
      }
    }
  }
  if (a.n_split == 1) return;
  if (a.cluster) {                             // each split joins some columns of all, in split order
    cluster_barrier();
    for (int col = split + a.n_split * threadIdx.x; col < G * 32; col += a.n_split * kThreads) {
      const int g = col >> 5;
      float2 ml[kMaxCluster];
      float4 s[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        const uint32_t p = remote(own + g * kPart, min(k, a.n_split - 1));
        ml[k] = ld_remote2(p);
        s[k] = ld_remote4(p + 16 + 16 * (col & 31));
      }
      float M = kNoRef, l = 0.f;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, ml[k].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k >= a.n_split || ml[k].y == 0.f) continue;   // saw no token
        const float f = exp2_neg(ml[k].x - M);
        l = fmaf(f, ml[k].y, l);
        acc.x = fmaf(f, s[k].x, acc.x);
        acc.y = fmaf(f, s[k].y, acc.y);
        acc.z = fmaf(f, s[k].z, acc.z);
        acc.w = fmaf(f, s[k].w, acc.w);
      }
      const float r = l == 0.f ? 0.f : 1.f / l;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * r, acc.y * r);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * r, acc.w * r);
      *reinterpret_cast<uint2*>(out + g * 128 + 4 * (col & 31)) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      if ((col & 31) == 0 && lse) lse[g] = lse_of(M, l);
    }
    cluster_barrier();                         // the others may still be reading this CTA's part
    return;
  }

  // ---- the last CTA of the pair joins the splits, in their order ----
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned t = atomicAdd(a.tickets + pair, 1u);
    last = t == (unsigned)a.n_split - 1u;
    if (last) a.tickets[pair] = 0;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float* sw = reinterpret_cast<float*>(smem);  // weights [split][G]
  float* sl = sw + kMaxSplits * G;             // [G] M, l
  // G * 32 columns of four channels; where threads are left, several share a
  // column, each a run of splits.  The first kFly parts of a run are on their way
  // before the weights are formed.
  constexpr int kCols = G * 32, kShare = kThreads / kCols, kFly = 16;
  const int col = threadIdx.x % kCols, sh = threadIdx.x / kCols;
  const int g = col >> 5, c4 = col & 31;
  const int run = (a.n_split + kShare - 1) / kShare, s0 = sh * run, s1 = min(s0 + run, a.n_split);
  auto part_of = [&](int s) {
    return __ldcg(reinterpret_cast<const float4*>(parts + ((size_t)s * G + g) * kPart + 4) + c4);
  };
  float4 fly[kFly];
#pragma unroll
  for (int u = 0; u < kFly; ++u) fly[u] = part_of(min(s0 + u, a.n_split - 1));
  if (warp < G) {
    const int g = warp;
    float M = kNoRef, l = 0.f;
    float m[kMaxSplits / 32], ll[kMaxSplits / 32];
#pragma unroll
    for (int u = 0; u < kMaxSplits / 32; ++u) {
      const int s = lane + 32 * u;
      m[u] = kNoRef;
      ll[u] = 0.f;
      if (s < a.n_split) {
        const float2 t = __ldcg(reinterpret_cast<const float2*>(parts + ((size_t)s * G + g) * kPart));
        m[u] = t.x;
        ll[u] = t.y;
      }
      M = fmaxf(M, m[u]);
    }
    M = warp_max_xor(M, 1);
#pragma unroll
    for (int u = 0; u < kMaxSplits / 32; ++u) {
      const float f = ll[u] == 0.f ? 0.f : exp2_neg(m[u] - M);
      l = fmaf(f, ll[u], l);
      sw[(lane + 32 * u) * G + g] = ll[u] == 0.f ? -1.f : f;   // below 0: a split that saw no token
    }
    l = warp_sum_xor(l, 1);
    if (lane == 0) {
      sl[g] = l;
      if (lse) lse[g] = lse_of(M, l);
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int s, const float4& p) {
    const float f = sw[s * G + g];
    if (!(f < 0.f)) {
      acc.x = fmaf(f, p.x, acc.x);
      acc.y = fmaf(f, p.y, acc.y);
      acc.z = fmaf(f, p.z, acc.z);
      acc.w = fmaf(f, p.w, acc.w);
    }
  };
#pragma unroll
  for (int u = 0; u < kFly; ++u)
    if (s0 + u < s1) add(s0 + u, fly[u]);
#pragma unroll 8
  for (int s = s0 + kFly; s < s1; ++s) add(s, part_of(s));
  float4* red = reinterpret_cast<float4*>(sl + ((G + 3) & ~3));
  if (kShare > 1) {
    red[threadIdx.x] = acc;
    __syncthreads();
  }
  if (sh == 0) {
#pragma unroll
    for (int u = 1; u < kShare; ++u) {
      const float4 t = red[u * kCols + col];
      acc.x += t.x;
      acc.y += t.y;
      acc.z += t.z;
      acc.w += t.w;
    }
    const float l = sl[g], f = l == 0.f ? 0.f : 1.f / l;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * f, acc.y * f), hi = __floats2bfloat162_rn(acc.z * f, acc.w * f);
    *reinterpret_cast<uint2*>(out + g * 128 + 4 * c4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// Splits per (sequence, KV head), from the host's bound on visible tiles (times by
// graph replay where below 15 us).
// - Up to two tiles per warp: none (256 tokens: 4.1 us, in two splits 6.2 through
//   memory; 512 tokens: 5.3 us, in four splits of a cluster 4.9).
// - Else a tile per warp at least, at most one wave of one CTA per SM where pairs are
//   few (8 pairs of 100,000 tokens: 37.9 us against 39.9 with two per SM, whose join
//   reads twice the parts), two per SM where that would leave SMs idle (128 pairs of
//   4,160 tokens: 29.3 us against 35.9), and about six waves for more pairs, so that
//   sequences of different lengths even out (512 pairs of 8k to 32k tokens: 398 us,
//   with four waves 408).
// - Where a cluster's worth of splits has up to two tiles per warp: no more than those
//   (2048 tokens: 5.5 us; in 16 splits, joined through memory, 7.1; beyond, 4096
//   tokens of 8 pairs: 8.2 so, 7.6 in 19).
// These are the times that the rule was made by; batches of 16 to 128 sequences of 512
// to 8,192 tokens, of which a warp may get a tile or two, were not measured.
int splits(const Pool& p, int B, long long max_len, int window, int n_sink) {
  long long tokens = max_len;
  if (window) tokens = std::min(tokens, (long long)window + n_sink + 2 * kTile);
  const long long tiles = (tokens + kTile - 1) / kTile, pairs = (long long)B * p.cfg.num_kv_heads, sms = p.sm_count;
  const long long want = sms >= 4 * pairs ? sms / pairs : (pairs <= sms ? 2 * sms / pairs : (12 * sms + pairs - 1) / pairs);
  if (tiles <= 2 * kWarps) return 1;
  const long long most = std::min<long long>((tiles + kWarps - 1) / kWarps, kMaxSplits);
  const long long n = std::max(1ll, std::min(want, most));
  return (int)(tiles <= 2 * kMaxCluster * kWarps ? std::min<long long>(n, kMaxCluster) : n);
}

// Clusters of n CTAs that the pool's device (the current one) holds at once.
constexpr int kDevices = 16;                                 // remembered: the first 16 devices
template <int G>
int resident_clusters(int device, int n) {
  static std::atomic<int> known[kDevices][kMaxCluster + 1];  // + 1; 0: not asked yet
  int have = device < kDevices ? known[device][n].load(std::memory_order_relaxed) : 0;
  if (have == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)n, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int count = 0;
    if (cudaOccupancyMaxActiveClusters(&count, decode_fp8_kernel<G>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      count = 0;
    }
    have = count + 1;
    if (device < kDevices) known[device][n].store(have, std::memory_order_relaxed);
  }
  return have - 1;
}

template <int G>
cudaError_t launch_t(const DecodeFp8Args& a, int device, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  const long long pairs = (long long)a.B * a.L.Hkv;
  DecodeFp8Args b = a;
  b.cluster = a.n_split > 1 && a.n_split <= kMaxCluster && pairs <= resident_clusters<G>(device, a.n_split);
  return launch_dependent(decode_fp8_kernel<G>, dim3((unsigned)(pairs * a.n_split)), kThreads, kSmem, s,
                          b.cluster ? a.n_split : 1, b);
}

}  // namespace

size_t decode_fp8_workspace(const Pool& p, int B, int max_len) {
  const int n = splits(p, B, max_len, 0, 0);
  return n == 1 ? 16 : (size_t)B * p.cfg.num_q_heads * n * kPart * sizeof(float);
}

// Fewer sequences are split further: the most that any batch up to B needs.
size_t decode_fp8_workspace_up_to(const Pool& p, int B, int max_len) {
  size_t most = 0;
  for (int b = 1; b <= B; ++b) most = std::max(most, decode_fp8_workspace(p, b, max_len));
  return most;
}

cudaError_t launch_decode_fp8(const Pool& p, const Fp8Store& f, int layer, int B, const AttnCall& c, cudaStream_t s) {
  DecodeFp8Args a{fp8_layer(p, f, layer), c, B, p.cfg.num_q_heads, splits(p, B, c.max_len, c.window, c.n_sink),
                  p.tickets + (size_t)layer * p.cfg.max_seqs * p.cfg.num_kv_heads, p.err,
                  p.test_wait_polls > 0 ? p.test_wait_polls : kPolls, p.test_stall_first_copy};
  switch (p.G) {
    case 1: return launch_t<1>(a, p.device, s);
    case 2: return launch_t<2>(a, p.device, s);
    case 4: return launch_t<4>(a, p.device, s);
    default: return launch_t<8>(a, p.device, s);
  }
}

}  // namespace kvint2
