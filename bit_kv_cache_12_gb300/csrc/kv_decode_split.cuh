// What the single-token attention kernels of the 8-bit and the 4-bit cache share: which
// tiles a query sees, and how the parts that warps, clusters and CTAs hold of a row's
// softmax are joined.
#pragma once

#include <atomic>

#include "kv_device.cuh"
#include "kv_fp8.h"

namespace kvint2 {

constexpr int kMaxSplits = 64;
constexpr int kMaxCluster = 8;                 // the portable cluster size
constexpr int kPart = 132;                     // floats of a partial head: M, l, 2 unused, 128 sums
constexpr float kNoRef = -3e38f;               // below every logit

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

// The last CTA of a pair to arrive joins the pair's splits, in their order.
template <int G, int kWarps, int kRoom>
__device__ __forceinline__ void join_through_memory(const float* parts, int n_split, unsigned* ticket, uint8_t* smem,
                                                    uint16_t* out, float* lse) {
  constexpr int kThreads = kWarps * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned t = atomicAdd(ticket, 1u);
    last = t == (unsigned)n_split - 1u;
    if (last) *ticket = 0;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float* sw = reinterpret_cast<float*>(smem);  // weights [split][G]
  float* sl = sw + kMaxSplits * G;             // [G] l
  float4* red = reinterpret_cast<float4*>(sl + ((G + 3) & ~3));
  float4* buf = red + kThreads;                // parts, as many as there is room for
  // G * 32 columns of four channels; where threads are left, several share a
  // column, each a run of splits.  The parts come to shared memory all at once
  // and the loops are short: loaded to registers by unrolled code, cold as it
  // is, 36 splits of four heads took 4.3 us instead of 2.5.
  constexpr int kCols = G * 32, kShare = kThreads / kCols, kQuads = G * kPart / 4;   // (16 bytes of a split)
  constexpr int kFit = (kRoom - kMaxSplits * G * 4 - 32 - kThreads * 16) / (kQuads * 16);
  static_assert(kFit >= 1, "a part fits");
  const int col = threadIdx.x % kCols, sh = threadIdx.x / kCols;
  const int g = col >> 5, c4 = col & 31;
  const int run = (n_split + kShare - 1) / kShare, s0 = sh * run, s1 = min(s0 + run, n_split);
  auto fetch = [&](int from, int to, int thread, int threads) {
    const float4* src = reinterpret_cast<const float4*>(parts) + (size_t)from * kQuads;
#pragma unroll 1
    for (int i = thread; i < (to - from) * kQuads; i += threads)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(buf + i)), "l"(src + i) : "memory");
  };
  constexpr int kForm = G < kWarps ? G : 0;    // warps that form the weights meanwhile
  if (warp >= kForm) fetch(0, min(kFit, n_split), threadIdx.x - 32 * kForm, kThreads - 32 * kForm);
  if (warp < G) {
    const int g = warp;
    float M = kNoRef, l = 0.f;
    float m[kMaxSplits / 32], ll[kMaxSplits / 32];
#pragma unroll
    for (int u = 0; u < kMaxSplits / 32; ++u) {
      const int s = lane + 32 * u;
      m[u] = kNoRef;
      ll[u] = 0.f;
      if (s < n_split) {
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
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int from = 0;;) {
    const int to = min(from + kFit, n_split);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll 2
    for (int s = max(s0, from); s < min(s1, to); ++s) {
      const float f = sw[s * G + g];
      const float4 p = buf[(s - from) * kQuads + g * (kPart / 4) + 1 + c4];
      if (f < 0.f) continue;
      acc.x = fmaf(f, p.x, acc.x);
      acc.y = fmaf(f, p.y, acc.y);
      acc.z = fmaf(f, p.z, acc.z);
      acc.w = fmaf(f, p.w, acc.w);
    }
    if (to == n_split) break;
    __syncthreads();
    from = to;
    fetch(from, min(from + kFit, n_split), threadIdx.x, kThreads);
  }
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

template <int G, int kWarps, int kRoom>
__device__ __noinline__ void join_apart(const float* parts, int n_split, unsigned* ticket, uint8_t* smem, uint16_t* out,
                                        float* lse) {
  join_through_memory<G, kWarps, kRoom>(parts, n_split, ticket, smem, out, lse);
}

// Joins what the warps of a CTA hold of the G heads of pair (b, h), then the splits of the
// pair, and writes the rows.  In shared memory, written and fenced by a barrier:
//   wo  [warp][head] sums of 128 channels, heads kHeadStride floats apart, channel c at at(c)
//   wm, wl  behind them, [warp][head] M and l (l = 0: saw no token)
// Parts are joined in the order of their warps and splits: the result does not depend on
// timing.  Splits of a cluster (n_split at most kMaxCluster) read one another's parts from
// shared memory; else the last CTA of the pair to arrive joins them through c.ws.  kRoom:
// bytes of smem that may be used.  kApart: that join is a function of its own, and the
// registers of the kernel's loops are allotted without it (the 4-bit kernel with G = 2, 4: 64 x
// 20,480 tokens 250 -> 245 us; the 8-bit one gains nothing and pays 0.4 us for the call).
template <int G, int kWarps, int kHeadStride, int kRoom, bool kApart, class Chan>
__device__ __forceinline__ void join_parts(const AttnCall& c, int Hq, int n_split, int cluster, unsigned* tickets,
                                           uint8_t* smem, int split, int pair, int b, int h, Chan at) {
  constexpr int kThreads = kWarps * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* wo = reinterpret_cast<float*>(smem);
  float* wm = wo + kWarps * G * kHeadStride;
  float* wl = wm + kWarps * G;
  uint16_t* out = static_cast<uint16_t*>(c.out) + ((size_t)b * Hq + h * G) * 128;
  float* lse = c.lse ? c.lse + (size_t)b * Hq + h * G : nullptr;
  float* parts = static_cast<float*>(c.ws) + (size_t)pair * n_split * G * kPart;
  float* own = wl + ((kWarps * G + 3) & ~3);   // cluster: this split's part
  for (int idx = threadIdx.x; idx < G * 128; idx += kThreads) {
    const int g = idx >> 7, ch = idx & 127;
    float M = kNoRef;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * G + g]);
    float l = 0.f, s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = wl[w * G + g] == 0.f ? 0.f : exp2_neg(wm[w * G + g] - M);
      l = fmaf(f, wl[w * G + g], l);
      if (wl[w * G + g] != 0.f) s = fmaf(f, wo[(w * G + g) * kHeadStride + at(ch)], s);
    }
    if (n_split == 1) {
      const float y = l == 0.f ? 0.f : s / l;
      out[g * 128 + ch] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      if (ch == 0 && lse) lse[g] = lse_of(M, l);
    } else {
      float* p = cluster ? own + g * kPart : parts + ((size_t)split * G + g) * kPart;
      p[4 + ch] = s;
      if (ch == 0) {
        p[0] = M;
        p[1] = l;
      }
    }
  }
  if (n_split == 1) return;
  if (cluster) {                             // each split joins some columns of all, in split order
    cluster_barrier();
    for (int col = split + n_split * threadIdx.x; col < G * 32; col += n_split * kThreads) {
      const int g = col >> 5;
      float2 ml[kMaxCluster];
      float4 s[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        const uint32_t p = remote(own + g * kPart, min(k, n_split - 1));
        ml[k] = ld_remote2(p);
        s[k] = ld_remote4(p + 16 + 16 * (col & 31));
      }
      float M = kNoRef, l = 0.f;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, ml[k].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k >= n_split || ml[k].y == 0.f) continue;   // saw no token
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

  if (kApart)
    join_apart<G, kWarps, kRoom>(parts, n_split, tickets + pair, smem, out, lse);
  else
    join_through_memory<G, kWarps, kRoom>(parts, n_split, tickets + pair, smem, out, lse);
}


// Clusters of n CTAs that the pool's device (the current one) holds at once.
constexpr int kDevices = 16;                                 // remembered: the first 16 devices
template <auto kernel, size_t kSmemBytes>
int resident_clusters(int device, int n, int threads) {
  static std::atomic<int> known[kDevices][kMaxCluster + 1];  // + 1; 0: not asked yet
  int have = device < kDevices ? known[device][n].load(std::memory_order_relaxed) : 0;
  if (have == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)n, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int count = 0;
    if (cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      count = 0;
    }
    have = count + 1;
    if (device < kDevices) known[device][n].store(have, std::memory_order_relaxed);
  }
  return have - 1;
}

}  // namespace kvint2
