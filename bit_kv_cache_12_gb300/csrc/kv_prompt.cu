// Causal attention over packed bf16 rows on the tcgen05 tensor cores.
//
// A row is a (query token, query head of the KV head) pair, so the G heads that share a KV
// head share its tiles: a block of 256 rows holds 256 / G tokens.  Per row, with base-2
// logits  x_j = scale log2(e) (q . k_j):
//   w_j = 2^(x_j - M),   out = sum_j w_j v_j / sum_j w_j.
// M is the first tile's maximum and moves only when a weight would pass 2^20, so that the
// accumulator is hardly ever rescaled.  The weights enter their product with V as bf16 (its
// operands have one type, and V is bf16): 8 bits relative to their own size, as many as the
// output has.  The denominator sums the fp32 weights.
//
// One CTA per SM: two tiles of 128 rows take turns, one in the tensor cores while the other
// is in the softmax.
//   warps 0-3, 4-7   softmax of a tile: a thread owns a row; S is read from tensor memory,
//                    the weights go back over it as bf16
//   warps 8-11       write an item's rows, while the softmax is at the next one
//   warp 12          issues the products: S = Q K^T from shared memory, O += P V with P from
//                    tensor memory and V token-major as it is stored
//   warp 13          walks the items
//   warp 14          loads q, K and V tiles (TMA)
//   warp 15          hands loaded tiles on to the issuer, after a look through the values of
//                    those that some row sees only in part
// Tensor memory: S0, S1 (P over them), O0, O1, 128 columns each.
// Hidden keys: a tile that some row sees only in part is masked by select after the product
// (a NaN in a hidden K row never enters).  Its values that are not finite are zeroed in
// shared memory, or a weight of zero would make them NaN, and their tokens are listed; a row
// that sees such a token looks at those tiles' values again at its end and sets the channels
// that are not finite to NaN.
// Few rows: the keys are split over several CTAs, whose normalised parts a second kernel
// joins by their log-sum-exp.
//
// Bound: the tensor cores.  A pass of both tiles over 128 keys is 2,048 clocks of products
// and takes some 2,700 (1.43 us), an item 7 us beyond its passes.  A call of 512 tokens (four
// passes) spends 4,600 clocks up to its first scores (1,900 of them to find its item, 1,700 to
// have q and K), 2,000 to 3,000 in each softmax, and 10,700 behind the last one: 2,900 in the last
// products, 6,300 in writing two tiles' rows.  One token takes 13,800 in all.  8192 tokens of 32
// + 8 heads 363 us where the clock holds (two dozen calls; 1.51 PFLOP/s, 0.77 of a large library
// product's rate), 394 in a long stream, 4 chunks of 518 to 2000 tokens under a window of 4096
// 490 (1.31) and 520, 512 tokens 14.1.  What lies between: the issuer's way from one group of
// products to the next (four products in the queue cover 256 of its 290 to 420 clocks), and an
// item's rows, read from tensor memory (2,700 clocks a tile), before its successor's first
// products.  A softmax of half the work took 1.36 us a pass, the products with V alone left
// out 1.07; an issuer for each tile made 8192 tokens take 463 us (both tiles' products
// interleave, and then both softmaxes wait), weights handed on in halves 5% more than 376,
// items overlapped in full 385.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "kv_fp4.h"
#include "kv_tc.cuh"

namespace kvint2 {

namespace {

constexpr int kRows = 128;                     // rows of a tile (M of a product)
constexpr int kKeys = 128;                     // keys of a tile
constexpr int kThreads = 16 * 32;              // four warpgroups
// registers per thread of the softmax warpgroups and of the two others: they share the
// launch's 128 each
constexpr int kSoftRegs = 176, kOtherRegs = 80;
static_assert(2 * kSoftRegs + 2 * kOtherRegs <= 4 * 128, "setmaxnreg.inc draws on the launch's registers");
constexpr int kPolls = 1 << 18;                // bound of a wait: a poll suspends for up to 3.7 us, so about a second
constexpr int kMaxSplits = 32;
constexpr int kPart = 132;                     // floats of a row's part: lse, 3 unused, 128 channels
constexpr float kNoRef = -3e38f;
constexpr float kRaise = 20.f;
constexpr int kStages = 2;                     // of K and of V (the issuer takes them in turns)

constexpr uint32_t kOffQ = 0;                  // two tiles
constexpr uint32_t kOffK = 2 * kOperand;
constexpr uint32_t kOffV = kOffK + kStages * kOperand;
constexpr uint32_t kOffOut = kOffV + kStages * kOperand;   // 4 KB for each writing warp
constexpr uint32_t kOffInfo = kOffOut + 4 * 4096;

constexpr int kItems = 4;                      // ring of items
constexpr int kLists = 8;                      // ring of passes

constexpr int kRing = 4;                       // of barriers that may run ahead of those who wait for them

// Barriers.  kData: V of a pass and K of the next (an item's first K comes with q).  kGo:
// all that the products of a pass wait for, a ring for each tile: P, and for tile 0 that the
// data are there; for tile 1 that the loader has seen its scores.  kSFull: a tile's scores of a
// pass; those of tile 1 also say that what came before them is done with, the products of the
// pass before and its values among it.  A wait looks at one bit of its barrier's phase, so no
// barrier may complete twice before everyone who waits for it has looked.
enum { kData = 0, kGo = kData + kStages, kLooked = kGo + 2 * kRing, kQFull = kLooked + kRing, kSFull = kQFull + 2,
       kOFull = kSFull + 2, kORead = kOFull + 2, kLast = kORead + 2, kDrain = kLast + 4, kCancel, kItem, kFree = kItem + kItems,
       kBars = kFree + kItems };

// An item: a block of rows and the key tiles they see.
enum { kKeyed = 0, kNoKeys = 1, kStop = 2 };   // rows with keys, rows that see none, no item
struct Work {
  int state;
  int s, h, c0, k0, m, n, row0, split;         // sequence, KV head, first q and k row, queries, keys, first row of the block
  int pos0;                                    // position of the sequence's query 0
  int first, keys;                             // position of the first row; keys from here on are hidden from every row
  int low, sinks, ns, w0, i0, i1;              // tile list: the first ns tiles, then from w0; this split's part of it
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : i - ns + w0; }
};

struct Shared {
  Work work[kItems];
  uint4 cancel;                                // what the scheduler answered
  uint64_t bars[kBars];
  uint32_t list[kLists][4];                    // of a pass that is seen in part: tokens with values that are not finite,
  uint32_t any[kLists];                        // and whether there are some
  float l[2][2][kRows];                        // of an item with keys (odd, even) and tile: each row's l,
  uint32_t poison[2][2][4];                    // and whether it sees a token listed before the last pass;
  int2 end[2];                                 // the last pass, and of those seen in part
  uint32_t tmem;
  int abort;
  int steps;                                   // items looked at so far
  int given;                                   // items published so far
  int taken[2];                                // blocks taken on but not published: the one at hand, and (when that one
                                               // never will be) the one that the scheduler had been asked for; else -1
  int next[4];                                 // writing warps, at their end: the item whose rows would have come next
};
constexpr uint32_t kSmem = kOffInfo + sizeof(Shared) + 1024;

struct PromptArgs {
  PromptCall c;
  int Hq, Hkv, G, shift, n_split, q_blocks;    // G = 2^shift: 1, 2, 4 or 8
  int* err;
  int polls;
  int stall;                                   // test hook: CTA 0 withholds its first item's last values
};

// kind::f16, fp32 accumulator, bf16 operands, M = N = 128; bit 16: B is MN-major
constexpr uint32_t kIdescQK =
    (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
constexpr uint32_t kIdescPV =
    (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(kIdescQK), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(kIdescPV), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int c, int h, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(h), "r"(row), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int c, int h, int row) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c), "r"(h), "r"(row)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Whether a sequence's rows [c0, c1) and [k0, k1) are ones, as many as it may have.  (Differences
// are taken of what is known to be in order: others could pass 32 bits.)
__device__ __forceinline__ bool rows_in_range(const PromptArgs& a, int c0, int c1, int k0, int k1) {
  return c0 >= 0 && c1 >= c0 && c1 - c0 <= a.c.max_q && c1 <= a.c.q_rows && k0 >= 0 && k1 >= k0 && k1 - k0 <= a.c.max_k &&
         k1 <= a.c.kv_rows;
}

// Item x of the grid; false where it has no rows (the whole warp calls this).
__device__ __forceinline__ bool find_work(const PromptArgs& a, int x, Work& w) {
  // blocks of a sequence from its last (most keys) to its first
  unsigned y = x;
  w.split = 0;
  if (a.n_split > 1) {
    w.split = y % a.n_split;
    y /= a.n_split;
  }
  w.h = y % a.Hkv;
  y /= a.Hkv;
  w.s = y % a.c.n_seqs;
  const int blk = a.q_blocks - 1 - (int)(y / a.c.n_seqs);
  w.c0 = a.c.cu_q[w.s];
  w.k0 = a.c.cu_k[w.s];
  const int c1 = a.c.cu_q[w.s + 1], k1 = a.c.cu_k[w.s + 1];
  if (!rows_in_range(a, w.c0, c1, w.k0, k1)) {
    if ((threadIdx.x & 31) == 0 && blk == 0 && w.split == 0 && w.h == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return false;
  }
  w.m = c1 - w.c0;
  w.n = k1 - w.k0;
  w.row0 = blk * 2 * kRows;
  if ((long long)w.row0 >= (long long)w.m * a.G) return false;
  w.pos0 = w.n - w.m;
  const int p_lo = w.pos0 + (w.row0 >> a.shift), p_hi = w.pos0 + min((w.row0 + 2 * kRows) >> a.shift, w.m) - 1;
  w.low = a.c.window ? max(p_lo - a.c.window + 1, 0) : 0;
  const int end = max(p_hi + 1, 0);
  w.first = p_lo;
  w.keys = end;
  w.sinks = a.c.window ? a.c.n_sink : 0;
  w.w0 = min(w.low, end) / kKeys;
  w.ns = min((min(w.sinks, end) + kKeys - 1) / kKeys, w.w0);
  const int total = w.ns + (end + kKeys - 1) / kKeys - w.w0;
  const int per = a.n_split > 1 ? (unsigned)(total + a.n_split - 1) / a.n_split : total;
  w.i0 = min(w.split * per, total);
  w.i1 = min(w.i0 + per, total);
  w.state = w.i0 < w.i1 ? kKeyed : kNoKeys;
  return true;
}

// Whether some row of the block sees the tile from key t0 on only in part.
__device__ __forceinline__ bool in_part(const PromptArgs& a, const Work& w, int t0) {
  return t0 + kKeys - 1 > w.first || (a.c.window && t0 < w.keys - a.c.window && t0 + kKeys > w.sinks);
}

// ---- loader (one warp) -----------------------------------------------------------

struct Maps {
  const CUtensorMap *q, *k, *v;
};

// The loads of an item: false where a wait ran out.  Pass g brings V of its own and K of the
// next pass, into stages g and g + 1 modulo two: free when the scores of pass g - 1 are
// complete, and the products of pass g - 2 with them.  K of pass g is there before that: only
// the loader's word that it has seen those scores holds back the next ones, of the same barrier
// (with a ring of barriers instead the softmax spilled more, 8192 tokens 2.5% slower).  q, g:
// items and passes loaded so far.
__device__ __forceinline__ bool load_item(const PromptArgs& a, const Maps& maps, const Work& w, bool withhold, uint8_t* sm,
                                          Shared* sh, const Waiter& wait, int& q, int& g) {
  const int lane = threadIdx.x & 31, tokens = kRows >> a.shift, h = w.h, k0 = w.k0, q0 = w.c0 + (w.row0 >> a.shift);
  const uint32_t base = smem_u32(sm);
  auto load = [&](uint32_t to, const CUtensorMap* map, int head, int row, int bar) {
    load_box(base + to, map, 0, head, row, sh->bars + bar);
    load_box(base + to + kOperand / 2, map, 64, head, row, sh->bars + bar);
  };
  for (int i = w.i0; i < w.i1; ++i, ++g) {
    const int stage = g % kStages, last = i + 1 == w.i1;
    if (i == w.i0) {                           // q, in the place of the item's before, whose last scores these are
      if (lane == 0) {
        for (int tile = 0; tile < 2; ++tile) {
          mbar_expect_tx(sh->bars + kQFull + tile, tile ? kOperand : 2 * kOperand);
          load(kOffQ + tile * kOperand, maps.q, h * a.G, q0 + tile * tokens, kQFull + tile);
          if (!tile) load(kOffK + stage * kOperand, maps.k, h, k0 + w.tile(i) * kKeys, kQFull);
        }
      }
      ++q;
    }
    if (withhold && last) return false;
    if (lane == 0) {
      mbar_expect_tx(sh->bars + kData + stage, last ? kOperand : 2 * kOperand);
      if (!last) load(kOffK + (g + 1) % kStages * kOperand, maps.k, h, k0 + w.tile(i + 1) * kKeys, kData + stage);
      load(kOffV + stage * kOperand, maps.v, h, k0 + w.tile(i) * kKeys, kData + stage);
    }
    if (!__all_sync(0xffffffffu, wait(sh->bars + kSFull + 1, g & 1))) {
      ++g;                                     // (its loads are on their way)
      return false;
    }
    if (lane == 0) arrive(sh->bars + kGo + kRing + g % kRing);
  }
  __syncwarp();
  return true;
}

__device__ __forceinline__ void load_tiles(const PromptArgs& a, const Maps& maps, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const int lane = threadIdx.x & 31;
  int q = 0, g = 0;
  for (int item = 0;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) break;
    const Work& w = sh->work[slot];
    if (w.state == kStop) break;
    if (w.state == kKeyed && !load_item(a, maps, w, a.stall && blockIdx.x == 0 && item == 0, sm, sh, wait, q, g)) break;
    if (lane == 0) arrive(sh->bars + kFree + slot);
    __syncwarp();
  }
  // whatever happened to those who wait for them: no load may land after the CTA has ended
#pragma unroll 1
  for (int i = max(g - kStages, 0); i < g; ++i) mbar_wait(sh->bars + kData + i % kStages, (i / kStages) & 1, kPolls);
#pragma unroll 1
  for (int i = 0; i < 2; ++i)
    if (q) mbar_wait(sh->bars + kQFull + i, (q - 1) & 1, kPolls);
}

// ---- loaded tiles, and the values of those seen in part (one warp) --------------------

__device__ __forceinline__ void look_through(const PromptArgs& a, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const int lane = threadIdx.x & 31;
  int g = 0, part = 0;                         // passes, and those that are seen in part
  for (int item = 0;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) return;
    const Work& w = sh->work[slot];
    if (w.state == kStop) return;
    if (w.state == kKeyed) {
      for (int i = w.i0; i < w.i1; ++i, ++g) {
        const int stage = g % kStages, t0 = w.tile(i) * kKeys;
        if (!__all_sync(0xffffffffu, wait(sh->bars + kData + stage, (g / kStages) & 1))) return;
        if (!in_part(a, w, t0)) {
          if (lane == 0) arrive(sh->bars + kGo + g % kRing);
          continue;
        }
        uint8_t* tile = sm + kOffV + stage * kOperand + lane * 128;
        uint32_t any = 0;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {          // a lane to a token
          uint8_t* row = tile + 32 * 128 * q;
          bool bad = false;
          // where some row may not see all 32 tokens
          if (t0 + 32 * q + 31 > w.first || (a.c.window && t0 + 32 * q < w.keys - a.c.window && t0 + 32 * q + 31 >= w.sinks)) {
            // sums of products with zero: NaN if one of the values is not finite
            __nv_bfloat162 n[4];
            const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = zero;
            auto add = [&](__nv_bfloat162& s, uint32_t x) { s = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&x), zero, s); };
#pragma unroll
            for (int c = 0; c < 16; ++c) {     // the swizzle: eight lanes read eight different banks
              const uint4 x = *reinterpret_cast<const uint4*>(row + (c >> 3) * (kOperand / 2) + (((c ^ lane) & 7) << 4));
              add(n[0], x.x);
              add(n[1], x.y);
              add(n[2], x.z);
              add(n[3], x.w);
            }
            const __nv_bfloat162 sum = __hadd2(__hadd2(n[0], n[1]), __hadd2(n[2], n[3]));
            bad = __hisnan(sum.x) || __hisnan(sum.y);
          }
          const uint32_t listed = __ballot_sync(0xffffffffu, bad);
          any |= listed;
          if (lane == 0) sh->list[g & (kLists - 1)][q] = listed;
          if (bad) {
#pragma unroll 1
            for (int c = 0; c < 64; ++c) {
              uint32_t* p = reinterpret_cast<uint32_t*>(row + (c >> 5) * (kOperand / 2)) + (c & 31);
              uint32_t x = *p;
              if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
              if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
              *p = x;
            }
          }
          __syncwarp();
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          sh->any[g & (kLists - 1)] = any;
          arrive(sh->bars + kLooked + part % kRing);
          arrive(sh->bars + kGo + g % kRing);
        }
        ++part;
      }
    }
    if (lane == 0) arrive(sh->bars + kFree + slot);
    __syncwarp();
  }
}

// ---- walker (one warp) -------------------------------------------------------------

// The items: this CTA's own, then those of CTAs that have not been launched yet, asked of
// the hardware's scheduler one ahead.
__device__ __forceinline__ void walk(const PromptArgs& a, const CUtensorMap* q, Shared* sh, const Waiter& wait) {
  const int lane = threadIdx.x & 31;
  auto ready = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(sh->bars + bar, parity)) != 0; };
  auto publish = [&](const Work& w, int item) -> bool {
    const int slot = item & (kItems - 1);
    if (item && w.state == kKeyed && lane < 4) // its q comes to the L2 cache while the items before are worked on
      prefetch_box(q, 64 * (lane & 1), w.h * a.G, w.c0 + (w.row0 >> a.shift) + (lane >> 1) * (kRows >> a.shift));
    if (item >= kItems && !ready(kFree + slot, (item / kItems - 1) & 1)) return false;
    if (lane == 0) {
      sh->work[slot] = w;
      sh->given = item + 1;
      sh->taken[0] = -1;
      arrive(sh->bars + kItem + slot);
    }
    __syncwarp();
    return true;
  };
  auto ask = [&](int steps) {
    if (lane == 0) {
      fence_async();
      mbar_expect_tx(sh->bars + kCancel, 16);
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
              smem_u32(&sh->cancel)),
          "r"(smem_u32(sh->bars + kCancel))
          : "memory");
      *reinterpret_cast<volatile int*>(&sh->steps) = steps;
    }
    __syncwarp();
  };
  int x = blockIdx.x, items = 0;
  bool ok = true;
  for (int asked = 0;; ++asked) {
    if (asked) ask(asked + 1);
    Work w;
    if (find_work(a, x, w)) ok = publish(w, items++);
    if (!asked) ask(1);                        // (after the first item, which everyone waits for)
    // the answer is waited for even when something failed: it is written to shared memory
    if (!__all_sync(0xffffffffu, mbar_wait(sh->bars + kCancel, asked & 1, kPolls))) {
      *reinterpret_cast<volatile int*>(wait.abort) = 1;
      return;
    }
    int got;
    asm volatile(
        "{ .reg .pred p; .reg .b128 h; ld.shared.b128 h, [%2]; "
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h; selp.b32 %0, 1, 0, p; "
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h; }"
        : "=r"(got), "+r"(x)
        : "r"(smem_u32(&sh->cancel))
        : "memory");
    if (lane == 0) sh->taken[!ok] = got ? x : -1;
    if (!ok) return;
    if (!__all_sync(0xffffffffu, got)) break;
  }
  Work stop{};
  stop.state = kStop;
  publish(stop, items);
}

// ---- product issuer (one warp) -----------------------------------------------------

// The whole warp runs this, in step, and one lane of it issues: addresses stay in uniform
// registers.  The loops are not unrolled: the code of the other warps passes through the
// same instruction cache, and a short loop stays in it.  The tensor cores take four products
// ahead (256 clocks), and a wait that the whole warp votes on takes some 150 of them: so
// there is one wait and one commit between two groups of products, both by the lane that
// issues.  After a wait that ran out it issues nothing more (`dead`); the others notice by
// the abort flag.
__device__ __forceinline__ void issue_products(const PromptArgs& a, uint32_t tmem, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const uint32_t base = smem_u32(sm);
  const uint64_t q0 = desc(base + kOffQ, 16), k0 = desc(base + kOffK, 16), v0 = desc(base + kOffV, kOperand / 2);
  bool dead = false;
  auto scores = [&](int tile, int stage) {     // the issuing lane
    uint64_t q = q0 + ((tile * kOperand) >> 4), k = k0 + ((stage * kOperand) >> 4);
    const uint32_t d = tmem + 128 * tile;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mma_ss(d, q + 2 * ks, k + 2 * ks, half | ks);
      q += (kOperand / 2) >> 4;
      k += (kOperand / 2) >> 4;
    }
    commit(sh->bars + kSFull + tile);
  };
  static_assert(kStages == 2, "the other stage is stage ^ 1");
  int g = 0, keyed = 0;                        // passes and items with keys so far
  for (int item = 0;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) return;
    const int state = sh->work[slot].state, passes = sh->work[slot].i1 - sh->work[slot].i0;
    if (state == kStop) return;
    if (state == kKeyed) {
      if (elect_one()) {
        dead = dead || !wait(sh->bars + kQFull, keyed & 1);
        fence_after();
        if (!dead) {
#pragma unroll 1
          for (int tile = 0; tile < 2; ++tile) {
            if (tile) dead = !wait(sh->bars + kQFull + 1, keyed & 1);
            if (!dead) scores(tile, g % kStages);
          }
        }
      }
      __syncwarp();
      if (elect_one()) {
#pragma unroll 1
        for (int it = 0; it < passes; ++it) {
          const int stage = (g + it) % kStages;
          const uint32_t parity = ((g + it) / kRing) & 1;
          uint64_t* go = sh->bars + kGo + (g + it) % kRing;
          const bool last = it + 1 == passes;
#pragma unroll 1
          for (int tile = 0; tile < 2; ++tile) {
            dead = dead || !wait(go + tile * kRing, parity);
            if (it == 0 && keyed) dead = dead || !wait(sh->bars + kORead + tile, (keyed - 1) & 1);
            fence_after();
            if (dead) continue;
            uint64_t v = v0 + ((stage * kOperand) >> 4);
            uint32_t p = tmem + 128 * tile;
            const uint32_t d = tmem + 256 + 128 * tile;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)   // 16 tokens: 8 columns of P, 16 rows of V
                mma_ts(d, p + 8 * ks, v + ((ks * 2048) >> 4), it | half | ks);
              p += 32;
              v += (4 * 2048) >> 4;
            }
            if (last)
              commit(sh->bars + kOFull + tile);
            else
              scores(tile, stage ^ 1);
          }
        }
      }
      __syncwarp();
      g += passes;
      ++keyed;
    }
    if (elect_one()) arrive(sh->bars + kFree + slot);
    __syncwarp();
  }
}

// ---- softmax (a thread owns a row) --------------------------------------------------

// Where row i of an item's block comes from and goes to.
struct Row {
  int token, hq;
  bool live;
  size_t qrow;
  __device__ __forceinline__ Row(const PromptArgs& a, const Work& w, int i) {
    const int row = w.row0 + i;                // of the sequence's rows
    token = row >> a.shift;
    hq = w.h * a.G + (row & (a.G - 1));
    live = token < w.m;
    qrow = ((size_t)w.c0 + token) * a.Hq + hq;
  }
};

struct RowOut {
  float M = kNoRef, l = 0.f;
  bool poison = false;                         // sees a token that is listed (before the last pass)
};

// The 32 keys from t0 on that the row at position pos sees.
__device__ __forceinline__ uint32_t sees(const PromptArgs& a, const Work& w, int pos, int t0) {
  uint32_t m = below(pos + 1 - t0, 0);
  if (a.c.window) m &= ~below(pos + 1 - a.c.window - t0, 0) | below(w.sinks - t0, 0);
  return m;
}
// Whether it sees a listed token of pass g, the part-th one of those seen in part, whose
// products have been issued (so that the wait only orders this after the look).
__device__ __forceinline__ bool poisoned(const PromptArgs& a, const Work& w, Shared* sh, int i, int t0, int g, int part) {
  mbar_wait(sh->bars + kLooked + part % kRing, (part / kRing) & 1, kPolls);
  if (!sh->any[g & (kLists - 1)]) return false;   // the usual case
  const int pos = w.pos0 + Row(a, w, i).token;
  uint32_t hit = 0;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) hit |= sh->list[g & (kLists - 1)][q] & sees(a, w, pos, t0 + 32 * q);
  return hit != 0;
}

// Scores of keys that this thread's row does not see: -inf (before the sign that scale may
// bring), in tensor memory.  A short loop beside the usual path: unrolled into it, it cost
// 1,500 clocks where it ran, cold as it is.
__device__ __forceinline__ void hide(const PromptArgs& a, const Work& w, uint32_t ts, int pos, int t0, bool minus) {
  const float none = minus ? INFINITY : -INFINITY;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t see = sees(a, w, pos, t0 + 32 * q);
    if (__all_sync(0xffffffffu, see == 0xFFFFFFFFu)) continue;
    float v[32];
    ld32(ts + 32 * q, v);
    settle(v);
    uint32_t u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = __float_as_uint((see >> i) & 1 ? v[i] : none);
    st16(ts + 32 * q, u);
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = __float_as_uint((see >> (16 + i)) & 1 ? v[16 + i] : none);
    st16(ts + 32 * q + 16, u);
  }
  wait_st();
}

// The passes of an item, up to its last weights.  g: the pass, counted over the CTA's
// items; left at the last one.  parts: those of them that are seen in part.
__device__ __forceinline__ bool softmax_rows(const PromptArgs& a, const Work& w, uint32_t trow, int tile, Shared* sh,
                                             const Waiter& wait, int& g, int& parts, RowOut& ro) {
  const uint32_t ts = trow + 128 * tile, to = trow + 256 + 128 * tile;
  const int i0 = tile * kRows + (threadIdx.x & 127), passes = w.i1 - w.i0;
  const bool minus = a.c.scale < 0.f;
  // above 0, so that a hidden key's -inf stays one
  const float cs = fmaxf(fabsf(a.c.scale) * 1.4426950408889634f, 1.17549435e-38f);
  int check = -1;                              // the pass before, where it was seen in part: its first key
  bool large = false;                          // this row's reference is
  for (int it = 0;; ++it, ++g) {
    const int t0 = w.tile(w.i0 + it) * kKeys;
    if (!__all_sync(0xffffffffu, wait(sh->bars + kSFull + tile, g & 1))) return false;
    fence_after();
    const bool part = in_part(a, w, t0);
    float c = cs;
    if (part) hide(a, w, ts, w.pos0 + Row(a, w, i0).token, t0, minus);
    float v[kKeys];
#pragma unroll
    for (int q = 0; q < 4; ++q) ld32(ts + 32 * q, v + 32 * q);
#pragma unroll
    for (int q = 0; q < 4; ++q) settle(v + 32 * q);
    if (minus) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) v[i] = -v[i];
    }
    float top[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      top[q] = fmaxf(v[32 * q], v[32 * q + 1]);
#pragma unroll
      for (int i = 2; i < 32; i += 2) top[q] = max3(top[q], v[32 * q + i], v[32 * q + i + 1]);
    }
    const float x = max3(fmaxf(top[0], top[1]), top[2], top[3]) * c;
    const bool raise = x - ro.M > kRaise;      // as a difference: where M is large, M + 20 is rounded by as much as that
    float d = -ro.M;
    if (__any_sync(0xffffffffu, raise || large)) {
      const float n = raise ? x : ro.M;
      const float f = exp2_neg(ro.M - n);
      ro.M = n;
      ro.l *= f;
      if (it > 0) {                            // the products so far are complete: S of this tile came after them
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float o[32];
          ld32(to + 32 * q, o);
          settle(o);
          uint32_t u[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * f);
          st16(to + 32 * q, u);
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[16 + i] * f);
          st16(to + 32 * q + 16, u);
        }
      }
      d = -n;
      large = large_reference(n);
      if (large) {                             // weights from the rounded logits; in here, where no usual pass comes by
#pragma unroll
        for (int i = 0; i < kKeys; ++i) v[i] = __fmul_rn(v[i], c) - n;
        c = 1.f;
        d = 0.f;
      }
    }
    const uint64_t c2 = f2(c, c), d2 = f2(d, d);
    uint64_t s0 = f2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t p[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float y0, y1;
        f2_split(f2_fma(f2(v[32 * q + 2 * i], v[32 * q + 2 * i + 1]), c2, d2), y0, y1);
        y0 = exp2_neg(y0);
        y1 = exp2_neg(y1);
        if (i & 1)
          s1 = f2_add(s1, f2(y0, y1));
        else
          s0 = f2_add(s0, f2(y0, y1));
        p[i] = pack_bf16(y0, y1);
      }
      st16(ts + 16 * q, p);
    }
    float sa, sb;
    f2_split(f2_add(s0, s1), sa, sb);
    ro.l += sa + sb;
    wait_st();
    fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive(sh->bars + kGo + tile * kRing + g % kRing);
    if (check >= 0) ro.poison |= poisoned(a, w, sh, i0, check, g - 1, parts - 1);   // while the products run
    check = part ? t0 : -1;
    parts += part;
    if (it + 1 == passes) return true;
  }
}

// A row's part of a split.
__device__ __forceinline__ float* part_of(const PromptArgs& a, const Work& w, const Row& r) {
  return static_cast<float*>(a.c.ws) + ((((size_t)w.s * a.c.max_q + r.token) * a.Hq + r.hq) * a.n_split + w.split) * kPart;
}

__device__ __forceinline__ void put_lse(const PromptArgs& a, const Work& w, const Row& r, float lse) {
  if (!r.live) return;
  if (a.n_split > 1)
    *part_of(a, w, r) = lse;
  else if (a.c.lse)
    a.c.lse[r.qrow] = lse;
}

// Channels 32 q .. of a row that sees listed tokens: a bit for each that some visible value
// makes not finite, from the tiles that are seen in part (in the others they went into the
// products as they are).
__device__ __forceinline__ uint32_t spoiled(const PromptArgs& a, const Work& w, int i, int q) {
  const int pos = w.pos0 + Row(a, w, i).token;
  uint32_t bits = 0;
#pragma unroll 1
  for (int it = w.i0; it < w.i1; ++it) {
    const int t0 = w.tile(it) * kKeys;
    if (!in_part(a, w, t0)) continue;
#pragma unroll 1
    for (int j = t0; j < min(t0 + kKeys, pos + 1); ++j) {
      if (a.c.window && j <= pos - a.c.window && j >= w.sinks) continue;
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.c.v) + (w.k0 + j) * a.c.v_stride +
                                                      w.h * 128 + 32 * q);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        const uint4 x = p[c];
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((u[e] & 0x7F80u) == 0x7F80u) bits |= 1u << (8 * c + 2 * e);
          if ((u[e] & 0x7F800000u) == 0x7F800000u) bits |= 2u << (8 * c + 2 * e);
        }
      }
    }
  }
  return bits;
}

// Rows of a tile, a thread to a row: its products times f to the output, or as a part of a
// split.  `stage`: 4 KB of shared memory for 64 channels of the warp's 32 rows, from which
// they are written 128 bytes at a time.  f 0: zeros, whatever the products are.  read: their
// barrier, arrived on once they are out of tensor memory.  Short loops: the code is cold
// whenever it runs (unrolled, a tile took 11,000 clocks; as it is 2,700).
__device__ __forceinline__ void write_rows(const PromptArgs& a, const Work& w, uint32_t to, uint8_t* stage, int row0, float f,
                                           uint64_t* read) {
  const int lane = threadIdx.x & 31, shift = a.shift;
  // to shared memory: this lane's row, 16-byte chunk c of row r at c ^ r % 8 (no bank
  // conflicts either way); from there: lane 8 u + c takes chunk c of rows 8 u + i
  uint8_t* put = stage + lane * 128;
  const uint32_t keep = f != 0.f ? 0xFFFFFFFFu : 0u;
  const uint8_t* get = stage + (lane >> 3) * 1024;
  const int token = (w.row0 + row0 + 8 * (lane >> 3)) >> shift, m = w.m;
  uint4* out = static_cast<uint4*>(a.c.out) + (((size_t)w.c0 + token) * a.Hq + w.h * a.G) * 16 + (lane & 7);
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
      float o[32];
      ld32(to + 64 * half + 32 * q, o);
      settle(o);
      const uint64_t ff = f2(f, f);
#pragma unroll
      for (int i = 0; i < 16; ++i) f2_split(f2_fma(f2(o[2 * i], o[2 * i + 1]), ff, f2(-0.f, -0.f)), o[2 * i], o[2 * i + 1]);
      if (a.n_split > 1) {
        const Row row(a, w, row0 + lane);
        if (row.live) {
          float* part = part_of(a, w, row) + 4 + 64 * half + 32 * q;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(__float_as_uint(o[i]) & keep);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(part + 4 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(put + (((4 * q + c) ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16(o[8 * c], o[8 * c + 1]) & keep, pack_bf16(o[8 * c + 2], o[8 * c + 3]) & keep,
                         pack_bf16(o[8 * c + 4], o[8 * c + 5]) & keep, pack_bf16(o[8 * c + 6], o[8 * c + 7]) & keep);
      }
    }
    if (half) {
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(read);
    }
    __syncwarp();
    if (a.n_split == 1) {
#pragma unroll 4
      for (int i = 0; i < 8; ++i)
        if (token + (i >> shift) < m)
          out[(size_t)((i >> shift) * a.Hq + (i & (a.G - 1))) * 16 + 8 * half] =
              *reinterpret_cast<const uint4*>(get + i * 128 + (((lane & 7) ^ i) << 4));
      __syncwarp();
    }
  }
}

// The channels of a row that some visible value makes not finite, over what was just written.
__device__ __forceinline__ void spoil_row(const PromptArgs& a, const Work& w, int i) {
  const Row row(a, w, i);
  if (!row.live) return;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
#pragma unroll 1
    for (uint32_t bits = spoiled(a, w, i, q); bits; bits &= bits - 1) {
      const int c = 32 * q + __ffs(bits) - 1;
      if (a.n_split > 1)
        part_of(a, w, row)[4 + c] = __uint_as_float(0x7FC00000u);
      else
        static_cast<uint16_t*>(a.c.out)[row.qrow * 128 + c] = 0x7FC0;
    }
  }
}

// The rows of every item (four warps).  Returns the first item whose rows were not written.
__device__ __forceinline__ int write_items(const PromptArgs& a, uint32_t tmem, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, m = 32 * warp + lane;
  int keyed = 0, item = 0;
  for (;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) break;
    const Work& w = sh->work[slot];
    if (w.state == kStop) break;
    const bool any = w.state == kKeyed;
    float f0 = 0.f, f1 = 0.f;                  // of this thread's rows of the two tiles
    const int rows = (w.m << a.shift) - w.row0 - 32 * warp;   // from this warp's first on
    uint32_t poison = 0;                       // whether they see a listed token
    if (any) {
      const int t0 = w.tile(w.i1 - 1) * kKeys;
      const bool part = in_part(a, w, t0);
#pragma unroll 1
      for (int tile = 0; tile < 2; ++tile) {
        if (!__all_sync(0xffffffffu, wait(sh->bars + kLast + 2 * (keyed & 1) + tile, (keyed >> 1) & 1))) return item;
        const float l = sh->l[keyed & 1][tile][m];
        f0 = f1;
        f1 = l != 0.f ? 1.f / l : 0.f;
        uint32_t hit = (sh->poison[keyed & 1][tile][warp] >> lane) & 1;
        // asked before the products are given back: so the looking warp is at most two passes
        // on, and the barrier of the last pass still in its phase
        if (part) hit |= poisoned(a, w, sh, tile * kRows + m, t0, sh->end[keyed & 1].x, sh->end[keyed & 1].y);
        poison |= hit << tile;
      }
    }
#pragma unroll 1
    for (int tile = 0; tile < 2; ++tile) {
      if (!any) {
        const Row row(a, w, tile * kRows + m);
        put_lse(a, w, row, -INFINITY);
        uint4* out = static_cast<uint4*>(a.c.out) + row.qrow * 16;
#pragma unroll 1
        for (int c = 0; c < 16 && row.live && a.n_split == 1; ++c) out[c] = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (!__all_sync(0xffffffffu, wait(sh->bars + kOFull + tile, keyed & 1))) return item;
      fence_after();
      if (tile * kRows >= rows) {              // none of this warp's exist (one token 8.5 -> 7.7 us; 512 13.9 -> 14.0)
        if (lane == 0) arrive(sh->bars + kORead + tile);
        continue;
      }
      write_rows(a, w, tmem + ((uint32_t)(32 * warp) << 16) + 256 + 128 * tile, sm + kOffOut + warp * 4096,
                 tile * kRows + 32 * warp, tile ? f1 : f0, sh->bars + kORead + tile);
    }
#pragma unroll 1
    for (int tile = 0; tile < 2; ++tile)
      if ((poison >> tile) & 1) spoil_row(a, w, tile * kRows + m);
    if (any) ++keyed;
    __syncwarp();
    if (lane == 0) arrive(sh->bars + kFree + slot);
  }
  return item;
}

// Rows of items that a CTA took on and did not get to before it gave up: not a number (in a
// split, the row's part: the join would read what the workspace held before).  first: the
// first item whose rows this warp has not written.
__device__ __forceinline__ void abandon(const PromptArgs& a, const Shared* sh, int first) {
  const int given = sh->given;
  const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll 1
  for (int item = first; item < given + 2; ++item) {
    Work w;
    if (item < given)
      w = sh->work[item & (kItems - 1)];
    else if (sh->taken[item - given] < 0 || !find_work(a, sh->taken[item - given], w))
      continue;
    if (w.state == kStop) return;
#pragma unroll 1
    for (int tile = 0; tile < 2; ++tile) {     // this thread's rows
      const Row row(a, w, tile * kRows + (threadIdx.x & 127));
      if (!row.live) continue;
      if (a.n_split > 1) {
        *part_of(a, w, row) = nan;
      } else {
        uint4* out = static_cast<uint4*>(a.c.out) + row.qrow * 16;
#pragma unroll 1
        for (int c = 0; c < 16; ++c) out[c] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        if (a.c.lse) a.c.lse[row.qrow] = nan;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(PromptArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Shared* sh = reinterpret_cast<Shared*>(sm + kOffInfo);
  const int warp = threadIdx.x >> 5;
  release_successor();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(sh->bars + kData + i, 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(sh->bars + kGo + i, 4 + 1);    // softmax warps, looking warp
      mbar_init(sh->bars + kGo + kRing + i, 4 + 1);   // softmax warps, loader
      mbar_init(sh->bars + kLooked + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh->bars + kQFull + i, 1);
      mbar_init(sh->bars + kSFull + i, 1);
      mbar_init(sh->bars + kOFull + i, 1);
      mbar_init(sh->bars + kORead + i, 4);
      mbar_init(sh->bars + kLast + i, 4);      // of odd and even items: the softmax may be one ahead of the rows
      mbar_init(sh->bars + kLast + 2 + i, 4);
    }
    mbar_init(sh->bars + kDrain, 1);
    mbar_init(sh->bars + kCancel, 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(sh->bars + kItem + i, 1);
      mbar_init(sh->bars + kFree + i, 8 + 4 + 3);       // softmax, writing warps, loader, issuer, looking warp
    }
    mbar_fence_init();
    sh->abort = 0;
    sh->steps = 0;
    sh->given = 0;
    sh->taken[0] = blockIdx.x;
    sh->taken[1] = -1;
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh->tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  after_predecessor();
  const uint32_t tmem = sh->tmem;
  const Waiter wait{&sh->abort, a.polls, &sh->steps};
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int tile = warp >> 2, lane = threadIdx.x & 31;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    int g = 0, parts = 0, keyed = 0;
    for (int item = 0;; ++item) {
      const int slot = item & (kItems - 1);
      if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) break;
      const Work& w = sh->work[slot];
      if (w.state == kStop) break;
      if (w.state == kKeyed) {
        RowOut ro;
        if (!softmax_rows(a, w, trow, tile, sh, wait, g, parts, ro)) break;
        sh->l[keyed & 1][tile][threadIdx.x & 127] = ro.l;
        const uint32_t poison = __ballot_sync(0xffffffffu, ro.poison);
        if (lane == 0) {
          sh->poison[keyed & 1][tile][warp & 3] = poison;
          if (warp == 0) sh->end[keyed & 1] = make_int2(g, parts - 1);
        }
        __syncwarp();
        if (lane == 0) arrive(sh->bars + kLast + 2 * (keyed & 1) + tile);
        put_lse(a, w, Row(a, w, tile * kRows + (threadIdx.x & 127)), lse_of(ro.M, ro.l));   // while the last products run
        ++g;
        ++keyed;
      }
      if (lane == 0) arrive(sh->bars + kFree + slot);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < 12) {
      const int next = write_items(a, tmem, sm, sh, wait);
      if ((threadIdx.x & 31) == 0) sh->next[warp - 8] = next;
    }
    if (warp == 12) issue_products(a, __shfl_sync(0xffffffffu, tmem, 0), sm, sh, wait);
    if (warp == 13) walk(a, &mq, sh, wait);
    if (warp == 14) load_tiles(a, {&mq, &mk, &mv}, sm, sh, wait);
    if (warp == 15) look_through(a, sm, sh, wait);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp >= 8 && warp < 12 && sh->abort) abandon(a, sh, sh->next[warp - 8]);
  if (warp == 12) {
    if (sh->abort) {                           // products may be in flight: wait (bounded) before giving back the memory
      if (elect_one()) {                       // the lane that issued them
        flag_error(a.err, KV_DEVERR_TIMEOUT);
        commit(sh->bars + kDrain);
        mbar_wait(sh->bars + kDrain, 0, kPolls);
      }
      __syncwarp();
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the splits of a row: a warp per row, four channels per lane.
__global__ void __launch_bounds__(256) prompt_join_kernel(PromptArgs a) {
  release_successor();
  after_predecessor();
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int hq = (int)(item % a.Hq);
  const long long t = item / a.Hq;
  const int s = (int)(t / a.c.max_q), i = (int)(t % a.c.max_q);
  if (s >= a.c.n_seqs) return;
  const int c0 = a.c.cu_q[s], c1 = a.c.cu_q[s + 1];
  if (!rows_in_range(a, c0, c1, a.c.cu_k[s], a.c.cu_k[s + 1]) || i >= c1 - c0) return;
  const float* part = static_cast<const float*>(a.c.ws) + (size_t)item * a.n_split * kPart;
  const float mine = lane < a.n_split ? part[(size_t)lane * kPart] : -INFINITY;
  const bool nan = __any_sync(0xffffffffu, isnan(mine));
  const float top = warp_max_xor(mine, 1);
  const float wt = mine == -INFINITY ? 0.f : expf(mine - top);
  const float sum = warp_sum_xor(wt, 1);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < a.n_split; ++k) {
    const float f = __shfl_sync(0xffffffffu, wt, k);
    if (__shfl_sync(0xffffffffu, mine, k) == -INFINITY) continue;   // saw no key
    const float4 p = *reinterpret_cast<const float4*>(part + (size_t)k * kPart + 4 + 4 * lane);
    acc.x = fmaf(f, p.x, acc.x);
    acc.y = fmaf(f, p.y, acc.y);
    acc.z = fmaf(f, p.z, acc.z);
    acc.w = fmaf(f, p.w, acc.w);
  }
  const float r = sum == 0.f ? 0.f : 1.f / sum;
  const size_t row = ((size_t)c0 + i) * a.Hq + hq;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.c.out) + row * 128 + 4 * lane) =
      make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
  if (a.c.lse && lane == 0)
    a.c.lse[row] = nan ? __uint_as_float(0x7FC00000u) : (sum == 0.f ? -INFINITY : top + logf(sum));
}

// of a sequence, at most; one where the bound is 0, which looks at the sequence's count
long long q_blocks(const Pool& p, int max_q) { return std::max(((long long)max_q * p.G + 2 * kRows - 1) / (2 * kRows), 1ll); }

// Splits of the keys: where the blocks of rows fill less than half of the SMs, as many as
// fit in one wave, of at least four tiles each.
int splits(const Pool& p, int n_seqs, int max_q, long long max_k, int window, int n_sink) {
  long long keys = max_k;
  if (window) keys = std::min(keys, (long long)window + n_sink + std::min<long long>(max_q, 2 * kRows / p.G) + 2 * kKeys);
  const long long tiles = (keys + kKeys - 1) / kKeys, blocks = q_blocks(p, max_q) * n_seqs * p.cfg.num_kv_heads;
  if (max_q == 0) return 1;
  return (int)std::max(1ll, std::min<long long>({p.sm_count / blocks, tiles / 4, kMaxSplits}));
}

// [rows][heads][128] bf16 as a tensor map of boxes of 64 channels of `heads` heads of `rows` rows
bool make_map(CUtensorMap* map, const void* base, int heads, long long rows, int64_t stride, int box_heads, int box_rows) {
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  const cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)std::max(rows, 1ll)};
  const cuuint64_t strides[2] = {256, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t prompt_workspace(const Pool& p, int n_seqs, int max_q, int max_k) {
  const int n = splits(p, n_seqs, max_q, max_k, 0, 0);
  return n == 1 ? 16 : (size_t)n_seqs * max_q * p.cfg.num_q_heads * n * kPart * sizeof(float);
}

// Fewer blocks of rows are split further: the most that any call up to these bounds needs.
// Only calls of up to half as many blocks as SMs are split; among those of as many blocks of
// queries the one with the most queries needs the most.
size_t prompt_workspace_up_to(const Pool& p, int n_seqs, int max_q, int max_k) {
  size_t most = 16;
  const int few = p.sm_count / 2;
  for (int b = 1; b <= std::min<long long>(few, q_blocks(p, max_q)); ++b)
    for (int s = 1; s <= std::min(few / b, n_seqs); ++s)
      most = std::max(most, prompt_workspace(p, s, std::min(max_q, b * 2 * kRows / p.G), max_k));
  return most;
}

cudaError_t launch_prompt(const Pool& p, const PromptCall& c, cudaStream_t s) {
  PromptArgs a{c, p.cfg.num_q_heads, p.cfg.num_kv_heads, p.G, __builtin_ctz(p.G), splits(p, c.n_seqs, c.max_q, c.max_k, c.window, c.n_sink),
               (int)q_blocks(p, c.max_q), p.err, p.test_wait_polls > 0 ? p.test_wait_polls : kPolls, p.test_stall_first_copy};
  const long long ctas = (long long)a.q_blocks * c.n_seqs * a.Hkv * a.n_split;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, c.q, a.Hq, c.q_rows, c.q_stride, a.G, kRows / a.G) ||
      !make_map(&mk, c.k, a.Hkv, c.kv_rows, c.k_stride, 1, kKeys) || !make_map(&mv, c.v, a.Hkv, c.kv_rows, c.v_stride, 1, kKeys))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(prompt_kernel, dim3((unsigned)ctas), kThreads, kSmem, s, 1, a, mq, mk, mv);
  if (e != cudaSuccess || a.n_split == 1) return e;
  return launch_dependent(prompt_join_kernel, dim3((unsigned)(((long long)c.n_seqs * c.max_q * a.Hq + 7) / 8)), 256, 0, s, 1, a);
}

}  // namespace kvint2
