// Single-token attention over the 4-bit cache, split over the cache.
//
// With code values k, v (e2m1), block scales sK, sV (e4m3), the layer's exponents and
// base-2 logits
//   x_j = scale log2(e) 2^eK sum_c q_c k_jc sK_j(c / 16),   w_j = 2^(x_j - M),
// a head's output is  2^eV sum_j w_j sV_j v_j / sum_j w_j.
//
// Both products are m16n8k16 tensor-core steps with the cached tile as the A operand and
// the (up to 8) query heads of the KV head as the 8 columns.  A code pair becomes an fp16
// register by one conversion.  The scales multiply the operand (code * scale has 6 bits and
// lies between 2^-10 and 2688: exact); which channels a step of K takes is free as long as
// q's rows agree, and with 32 neighbouring ones to a lane it needs two scales per token.  Of
// V the 16 rows of A are 16 channels of one block, a scale for each token.  (On the weights
// instead, the other operand, V's scales take half the multiplications and 64 sequences of 8k
// to 32k 295 us instead of 298; but a product below fp16's range is lost, 2^-19 of the largest
// weight where the scales are smallest, and tails of thousands of tokens with it.)  q
// enters as fp16 scaled per head by a power of two (largest element in [2^14, 2^15)): exact
// for bf16's 8 bits down to 2^-32 of it.  The weights are rounded to fp16; M lags so that the
// largest is between 2^7 and 2^15, and weights below 2^-32 of the largest are dropped.
//
// Bound: the cache's bytes (144 per token and KV head) for batches, latency for one short
// sequence, between them the instructions that turn codes into operands (issue slots 66% in
// use, tensor pipe 31%).  A warp takes two tiles at a step, copied whole (TMA, 4608 bytes)
// two steps ahead, so that one tile's conversions run beside the other's products: with one
// tile 64 sequences of 20,480 tokens took 317 us, with two 255.  Measured: 1024 tokens of 2
// KV heads 4.8 us (5.5 with the host's part), 16,384 tokens of 8 9.7, 100,000 26.5 (115 MB,
// 4.4 TB/s), 64 ragged sequences of 8k to 32k 298 us (1745 MB, 5.9 TB/s, 0.87 of a plain copy);
// under a window of 4096 with 64 first tokens 1 x 131,072 tokens of 8 KV heads 7.1, 16 of them
// 21.2 (77 MB, 3.6 TB/s).
#include <algorithm>

#include "kv_decode_split.cuh"
#include "kv_fp4.h"

namespace kvint2 {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 2 * kTile;               // tokens of a step: two tiles
constexpr uint32_t kUnitBytes = 2 * kFp4TileBytes;
constexpr int kStages = 3;                     // units in flight per warp
constexpr int kPolls = 1 << 18;                // bound of a copy's wait: a poll suspends for up to 3.7 us, so about a second
constexpr float kRaise = 15.f, kHead = 7.f;    // M moves when x > M + 15, to the largest x - 7
constexpr uint32_t kRing = kWarps * kStages * kUnitBytes;
constexpr uint32_t kSmem = kRing + kWarps * kStages * 8;
// Results of the warps in shared memory (over the ring): heads 136 floats apart, so that a
// half warp's pairs of channels fall into different banks.
constexpr int kHeadStride = 136;
static_assert(kWarps * 8 * (kHeadStride + 2) * 4 + 8 * kPart * 4 <= (int)kRing, "the results fit over the ring");
static_assert(kMaxSplits * 8 * 4 + 64 + kThreads * 16 <= (int)kRing, "and the join's weights and sums");

struct DecodeFp4Args {
  Fp4Layer L;
  AttnCall c;
  int B, Hq, n_split;
  unsigned* tickets;
  int* err;
  int polls;
  int stall;                                   // test hook: warp 0 of CTA 0 never starts its first copy
  int cluster;                                 // the splits of a pair are a cluster
};

// The units a query at position n - 1 sees: the first `ns`, then those from w0 on.
struct Units {
  int n, low, sinks, ns, w0, total;
  __device__ __forceinline__ Units(int len, int window, int n_sink) {
    n = len;
    low = window ? max(len - window, 0) : 0;
    sinks = window ? min(n_sink, len) : 0;
    w0 = low / kUnit;
    ns = min((sinks + kUnit - 1) / kUnit, w0);
    total = ns + (len + kUnit - 1) / kUnit - w0;
  }
  __device__ __forceinline__ int unit(int i) const { return i < ns ? i : i - ns + w0; }
  // bit t: token t of the unit is visible
  __device__ __forceinline__ uint32_t mask(int unit) const {
    const int t0 = unit * kUnit;
    auto below = [&](int j) { return j <= t0 ? 0u : (j - t0 >= kUnit ? 0xFFFFFFFFu : (1u << (j - t0)) - 1u); };
    return below(n) & (~below(low) | below(sinks));
  }
};

// The four code pairs of a word as fp16 pairs.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{ .reg .b8 p, q, r, s; mov.b32 {p, q, r, s}, %4; cvt.rn.f16x2.e2m1x2 %0, p; cvt.rn.f16x2.e2m1x2 %1, q; "
      "cvt.rn.f16x2.e2m1x2 %2, r; cvt.rn.f16x2.e2m1x2 %3, s; }"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) { return h2_as_u32(__hmul2(u32_as_h2(a), u32_as_h2(b))); }

template <int G>
__global__ void __launch_bounds__(kThreads, 2) decode_fp4_kernel(DecodeFp4Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  uint8_t* ring = smem + warp * kStages * kUnitBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kRing) + warp * kStages;
  if (lane < kStages) mbar_init(bar + lane, 1);
  mbar_fence_init();
  __syncwarp();
  release_successor();
  after_predecessor();

  const int split = blockIdx.x % a.n_split, pair = blockIdx.x / a.n_split;
  const int h = pair % a.L.Hkv, b = pair / a.L.Hkv;
  int n = a.c.seq_len[b];
  // lane (r, j) holds head r, channels 32 j ..; on its way with the length
  uint32_t qf[16];
  {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.c.q) +
                                                    ((size_t)b * a.Hq + h * G + (r < G ? r : 0)) * 128 + 32 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = q[i];
      qf[4 * i] = x.x, qf[4 * i + 1] = x.y, qf[4 * i + 2] = x.z, qf[4 * i + 3] = x.w;
    }
  }
  if (n < 0 || n > a.c.max_len) {
    if (split == 0 && threadIdx.x == 0) flag_error(a.err, KV_DEVERR_LENGTH);
    n = min(max(n, 0), a.c.max_len);
  }
  const Units un(n, a.c.window, a.c.n_sink);
  const int per = (un.total + a.n_split - 1) / a.n_split;
  const int i0 = split * per, count = max(min(per, un.total - i0), 0);
  const int mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;   // units i0 + warp, + kWarps, ..
  const int32_t* pt = a.c.pt + (size_t)b * a.c.max_pages;
  const bool wide = a.L.P == kUnit;            // a unit is a page, not two

  // The warp's k-th unit: what is visible of it, and the stored index of its tiles (below
  // 2^31: 2304 bytes each; -1: not visible, or behind a bad page id).  Page ids are read a
  // batch of 32 units ahead and not looked at before their turn (no load below waits for
  // another where it is issued); those of hidden tiles are not looked at at all.
  struct Batch {
    uint32_t vis;
    int pid0, pid1;
  };
  auto batch_of = [&](int k) -> Batch {
    Batch x;
    const int u = un.unit(i0 + warp + k * kWarps);
    x.vis = k < mine ? un.mask(u) : 0u;
    x.pid0 = pt[x.vis & 0xFFFFu ? (wide ? u : 2 * u) : 0];
    x.pid1 = pt[x.vis >> 16 ? (wide ? u : 2 * u + 1) : 0];
    return x;
  };
  auto tile_of = [&](uint32_t vis, int pid, int second) -> int {
    if (!vis) return -1;
    if (pid < 0 || pid >= a.L.num_pages) {
      flag_error(a.err, KV_DEVERR_PAGE_ID);
      return -1;
    }
    const int t = pid * a.L.Hkv + h;
    return wide ? 2 * t + second : t;
  };
  const uint64_t policy = l2_evict_first_policy();
  auto issue = [&](int stage, int t0, int t1) {  // lane 0
    uint8_t* to = ring + stage * kUnitBytes;
    mbar_expect_tx(bar + stage, (t0 >= 0 ? kFp4TileBytes : 0) + (t1 >= 0 ? kFp4TileBytes : 0));
    if (t0 >= 0) bulk_g2s_hint(to, a.L.tiles + (size_t)t0 * kFp4TileBytes, kFp4TileBytes, bar + stage, policy);
    if (t1 >= 0)
      bulk_g2s_hint(to + kFp4TileBytes, a.L.tiles + (size_t)t1 * kFp4TileBytes, kFp4TileBytes, bar + stage, policy);
  };
  // lane l knows the l-th unit of the current 32 and the page ids of the next
  Batch ahead = batch_of(lane);
  int cur0 = tile_of(ahead.vis & 0xFFFFu, ahead.pid0, 0), cur1 = tile_of(ahead.vis >> 16, ahead.pid1, 1);
  uint32_t vis_now = ahead.vis & ((cur0 >= 0 ? 0xFFFFu : 0u) | (cur1 >= 0 ? 0xFFFF0000u : 0u)), whole = 0;
  int next0 = -1, next1 = -1;
  uint32_t vis_next = 0;
  ahead = batch_of(32 + lane);
#pragma unroll
  for (int k = 0; k < kStages; ++k) {
    const int t0 = __shfl_sync(0xffffffffu, cur0, k), t1 = __shfl_sync(0xffffffffu, cur1, k);
    if (lane != 0 || k >= mine) continue;
    if (a.stall && k == 0 && blockIdx.x == 0 && warp == 0)
      mbar_expect_tx(bar, kFp4TileBytes);
    else
      issue(k, t0, t1);
  }

  // q as the B operand: scaled per head by a power of two, fp16
  float cs0, cs1;
  {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (r >= G) qf[i] = 0;                   // columns without a head
      top = max(top, max(qf[i] & 0x7FFFu, (qf[i] >> 16) & 0x7FFFu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int up = min(14 - ((int)(top >> 7) - 127), 126);
    const float mul = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : pow2i(up);   // not finite: NaN
#pragma unroll
    for (int i = 0; i < 16; ++i) qf[i] = pack_f16(bf16lo(qf[i]) * mul, bf16hi(qf[i]) * mul);
    const float cs = a.c.scale * 1.4426950408889634f * pow2i(a.L.k_exp) * pow2i(-up);
    cs0 = __shfl_sync(0xffffffffu, cs, 8 * j);          // heads 2j, 2j + 1
    cs1 = __shfl_sync(0xffffffffu, cs, 8 * j + 4);
  }

  float M0 = kNoRef, M1 = kNoRef, l0 = 0.f, l1 = 0.f;
  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  bool ok = true;
  int k = 0, stage = 0, phase = 0;
  for (; k < mine; ++k) {
    if ((k & 31) == 0) {                       // the next 32: their page ids have been on the way since the last batch
      if (k) {
        cur0 = next0;
        cur1 = next1;
        vis_now = vis_next;
      }
      next0 = tile_of(ahead.vis & 0xFFFFu, ahead.pid0, 0);
      next1 = tile_of(ahead.vis >> 16, ahead.pid1, 1);
      vis_next = ahead.vis & ((next0 >= 0 ? 0xFFFFu : 0u) | (next1 >= 0 ? 0xFFFF0000u : 0u));
      ahead = batch_of(k + 64 + lane);
      whole = __ballot_sync(0xffffffffu, vis_now == 0xFFFFFFFFu);
    }
    // the lanes vote: a copy that lands just as the limit runs out must not part them
    if (!__all_sync(0xffffffffu, mbar_wait(bar + stage, phase, a.polls))) {
      ok = false;
      break;
    }
    const uint8_t* st = ring + stage * kUnitBytes;
    float x[2][4];                             // per tile: token r heads 2j, 2j + 1, then token r + 8
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* tile = st + t * kFp4TileBytes;
      const uint4 ka = *reinterpret_cast<const uint4*>(tile + r * 64 + j * 16);
      const uint4 kb = *reinterpret_cast<const uint4*>(tile + (r + 8) * 64 + j * 16);
      const uint32_t sa = cvt_lo(*reinterpret_cast<const uint16_t*>(tile + kFp4KScale + r * 8 + j * 2));
      const uint32_t sb = cvt_lo(*reinterpret_cast<const uint16_t*>(tile + kFp4KScale + (r + 8) * 8 + j * 2));
      float acc[2][4] = {};
#pragma unroll
      for (int half = 0; half < 2; ++half) {   // channels 32 j + 16 half ..: one scale for each token
        const uint32_t ma = __byte_perm(sa, sa, half ? 0x3232 : 0x1010), mb = __byte_perm(sb, sb, half ? 0x3232 : 0x1010);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t a0, a2, a4, a6, a1, a3, a5, a7;
          codes4((&ka.x)[2 * half + w], a0, a2, a4, a6);
          codes4((&kb.x)[2 * half + w], a1, a3, a5, a7);
          const int s = 4 * half + 2 * w;
          mma_f16(acc[half], mul2(a0, ma), mul2(a1, mb), mul2(a2, ma), mul2(a3, mb), qf[2 * s], qf[2 * s + 1]);
          mma_f16(acc[half], mul2(a4, ma), mul2(a5, mb), mul2(a6, ma), mul2(a7, mb), qf[2 * s + 2], qf[2 * s + 3]);
        }
      }
      x[t][0] = (acc[0][0] + acc[1][0]) * cs0;
      x[t][1] = (acc[0][1] + acc[1][1]) * cs1;
      x[t][2] = (acc[0][2] + acc[1][2]) * cs0;
      x[t][3] = (acc[0][3] + acc[1][3]) * cs1;
    }
    uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
    if (!((whole >> (k & 31)) & 1)) {          // hidden tokens: no weight, and scales of zero
      const uint32_t vis = __shfl_sync(0xffffffffu, vis_now, k & 31);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t v = vis >> (16 * t);
        if (!((v >> r) & 1)) x[t][0] = x[t][1] = -INFINITY;
        if (!((v >> (r + 8)) & 1)) x[t][2] = x[t][3] = -INFINITY;
        const uint32_t lo = (v >> (2 * j)) & 3u, hi = (v >> (2 * j + 8)) & 3u;
        keep[t] = (lo & 1 ? 0xFFu : 0u) | (lo & 2 ? 0xFF00u : 0u) | (hi & 1 ? 0xFF0000u : 0u) | (hi & 2 ? 0xFF000000u : 0u);
      }
    }
    // as differences: where M is large, M + 15 is rounded by as much as that
    const float t0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
    const float t1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
    if (__any_sync(0xffffffffu, fmaxf(t0 - M0, t1 - M1) > kRaise)) {
      const float u0 = warp_max_xor(t0, 4), u1 = warp_max_xor(t1, 4);
      const float n0 = u0 - M0 > kRaise ? u0 - kHead : M0, n1 = u1 - M1 > kRaise ? u1 - kHead : M1;
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
    }
    uint32_t p[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float w0 = exp2_neg(x[t][0] - M0), w1 = exp2_neg(x[t][1] - M1);
      const float w2 = exp2_neg(x[t][2] - M0), w3 = exp2_neg(x[t][3] - M1);
      l0 += w0 + w2;
      l1 += w1 + w3;
      p[t][0] = movmatrix_t(pack_f16(w0, w1));
      p[t][1] = movmatrix_t(pack_f16(w2, w3));
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* tile = st + t * kFp4TileBytes;
#pragma unroll
      for (int q = 0; q < 2; ++q) {            // blocks 4 q ..: channels 16 i + 2 r, 16 i + 2 r + 1 of block i
        const uint4 v = *reinterpret_cast<const uint4*>(tile + kFp4V + 512 * q + lane * 16);
        const uint4 g = *reinterpret_cast<const uint4*>(tile + kFp4VScale + j * 32 + 16 * q);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t v0, v1, v2, v3;
          codes4((&v.x)[w], v0, v1, v2, v3);
          const uint32_t s = (&g.x)[w] & keep[t], lo = cvt_lo(s), hi = cvt_hi(s);
          mma_f16(o[4 * q + w], mul2(v0, lo), mul2(v1, lo), mul2(v2, hi), mul2(v3, hi), p[t][0], p[t][1]);
        }
      }
    }
    __syncwarp();
    const int kn = k + kStages;
    if (kn < mine) {
      const bool same = (kn >> 5) == (k >> 5);
      const int u0 = __shfl_sync(0xffffffffu, same ? cur0 : next0, kn & 31);
      const int u1 = __shfl_sync(0xffffffffu, same ? cur1 : next1, kn & 31);
      if (lane == 0) issue(stage, u0, u1);
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

  // ---- the warps' results -> the CTA's, the pair's ----
  __syncthreads();                             // every warp is done with its ring
  float* wo = reinterpret_cast<float*>(smem);
  float* wm = wo + kWarps * G * kHeadStride;   // [warp][head] M, then l
  float* wl = wm + kWarps * G;
  l0 = warp_sum_xor(l0, 4);
  l1 = warp_sum_xor(l1, 4);
  const float ve = pow2i(a.L.v_exp);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int g = 2 * j + u;
    if (g < G) {
      float* d = wo + (warp * G + g) * kHeadStride + 2 * r;
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<float2*>(d + 16 * i) = make_float2(o[i][u] * ve, o[i][2 + u] * ve);
      if (r == 0) {
        wm[warp * G + g] = u ? M1 : M0;
        wl[warp * G + g] = u ? l1 : l0;
      }
    }
  }
  __syncthreads();
  // G = 8 has the registers for the join within (16 x 16,384 tokens 60.4 us, apart 62.0), G = 2 and 4
  // do not (G = 2: 59.5, apart 58.2)
  join_parts<G, kWarps, kHeadStride, (int)kRing, G < 8>(a.c, a.Hq, a.n_split, a.cluster, a.tickets, smem, split, pair, b,
                                                        h, [](int c) { return c; });
}

// Shared memory of which an SM has room for one CTA: where there are no more CTAs than SMs,
// each gets one to itself (the scheduler puts two on some and leaves others idle: 144 CTAs
// of 8 pairs of 16,384 tokens took 12.8 us, 152 9.8).
constexpr uint32_t kSmemAlone = 120 << 10;
static_assert(kSmem <= kSmemAlone, "room for one");
uint32_t smem_of(const Pool& p, long long ctas) { return ctas <= p.sm_count ? kSmemAlone : kSmem; }

// Microseconds that a call takes with each (sequence, KV head) pair in n splits of `units`
// units, by graph replay.  A step of eight warps takes 1.0 us where an SM has one CTA and
// 1.75 where it has two, which also start 1 us later (8 pairs of 100,000 tokens in 19 splits
// 27.9 us, in 38 25.9; of 32,768 13.2 and 14.1).  Up to two CTAs per SM all run at once;
// more come in waves, with 5.5 us for the start and end of each and an uneven last one (512
// pairs of 20,480 tokens: 263 us in one split, 247 in two, 255 in three; of 8,192: 110, 115
// and 120).  A join inside a cluster (up to 8 splits) costs 1.8 us, through memory 2.6 and
// 0.045 for each split (1024 tokens of 2 pairs: 4.8 us in 8 splits, 6.2 in 9, 6.8 in one).
// What the largest length of a batch costs, so that shorter ones are even with it.
double cost_of(const Pool& p, long long pairs, long long units, int n) {
  const long long ctas = pairs * n, sms = p.sm_count;
  const double steps = (double)units / n / kWarps;
  const double join = n == 1 ? 0. : (n <= kMaxCluster ? 1.8 : 2.6 + 0.045 * n);
  if (ctas <= sms) return join + 1.0 * steps;
  if (ctas <= 2 * sms) return join + 1.75 * steps + 1.;
  return join + (double)ctas / (2 * sms) * (1.75 * steps + 5.5) + 0.42 * steps;
}

// More than one split only up to so many CTAs: what the workspace is sized by.
long long most_ctas(const Pool& p) { return 16ll * p.sm_count; }
int most_splits(const Pool& p, long long pairs, long long units) {
  return (int)std::max(1ll, std::min<long long>({kMaxSplits, units, most_ctas(p) / pairs}));
}

template <int G>
cudaError_t launch_t(const DecodeFp4Args& a, const Pool& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(decode_fp4_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemAlone);
  if (e != cudaSuccess) return e;
  const long long pairs = (long long)a.B * a.L.Hkv;
  if (pairs * a.n_split > INT32_MAX) return cudaErrorInvalidValue;
  DecodeFp4Args b = a;                         // (b.cluster is 0)
  uint32_t smem = smem_of(p, pairs * a.n_split);
  if (a.n_split > 1 && a.n_split <= kMaxCluster) {
    // fewer clusters of CTAs that have an SM to themselves fit than of others
    if (smem == kSmemAlone && pairs > resident_clusters<decode_fp4_kernel<G>, kSmemAlone>(p.device, a.n_split, kThreads)) smem = kSmem;
    b.cluster = smem == kSmemAlone || pairs <= resident_clusters<decode_fp4_kernel<G>, kSmem>(p.device, a.n_split, kThreads);
  }
  return launch_dependent(decode_fp4_kernel<G>, dim3((unsigned)(pairs * a.n_split)), kThreads, smem, s,
                          b.cluster ? a.n_split : 1, b);
}

}  // namespace

// From the host's bound on visible tokens.
int decode_fp4_splits(const Pool& p, int B, int max_len, int window, int n_sink) {
  long long tokens = max_len;
  if (window) tokens = std::min(tokens, (long long)window + n_sink + 2 * kUnit);
  const long long units = (tokens + kUnit - 1) / kUnit, pairs = (long long)B * p.cfg.num_kv_heads;
  int best = 1;
  double least = cost_of(p, pairs, units, 1);
  for (int n = 2, most = most_splits(p, pairs, units); n <= most; ++n) {
    const double c = cost_of(p, pairs, units, n);
    if (c < least) {
      least = c;
      best = n;
    }
  }
  return best;
}

size_t decode_fp4_workspace(const Pool& p, int B, int n_split) {
  return n_split == 1 ? 16 : (size_t)B * p.cfg.num_q_heads * n_split * kPart * sizeof(float);
}

// What any call needs of up to B sequences of up to max_len tokens, whatever its window.
size_t decode_fp4_workspace_up_to(const Pool& p, int B, int max_len) {
  const long long units = ((long long)max_len + kUnit - 1) / kUnit, pairs = (long long)B * p.cfg.num_kv_heads;
  const long long parts = std::min(most_ctas(p), pairs * std::min<long long>(kMaxSplits, units));
  return std::max<size_t>(16, (size_t)parts * p.G * kPart * sizeof(float));
}

cudaError_t launch_decode_fp4(const Pool& p, const Fp4Layer& L, int layer, int B, int n_split, const AttnCall& c,
                              cudaStream_t s) {
  DecodeFp4Args a{L, c, B, p.cfg.num_q_heads, n_split,
                  p.tickets + (size_t)layer * p.cfg.max_seqs * p.cfg.num_kv_heads, p.err,
                  p.test_wait_polls > 0 ? p.test_wait_polls : kPolls, p.test_stall_first_copy};
  switch (p.G) {
    case 1: return launch_t<1>(a, p, s);
    case 2: return launch_t<2>(a, p, s);
    case 4: return launch_t<4>(a, p, s);
    default: return launch_t<8>(a, p, s);
  }
}

}  // namespace kvint2
