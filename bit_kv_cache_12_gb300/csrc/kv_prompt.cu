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
//                    the weights go back over it as bf16; then this item's rows
//   warps 8-11       look through the values of tiles that some row sees only in part
//   warp 12          issues the products: S = Q K^T from shared memory, O += P V with P from
//                    tensor memory and V token-major as it is stored
//   warp 13          walks the items; warp 14 loads q, K and V tiles (TMA); warp 15 idles
// Tensor memory: S0, S1 (P over them), O0, O1, 128 columns each.
// Hidden keys: a tile that some row sees only in part is masked by select after the product
// (a NaN in a hidden K row never enters).  Its values that are not finite are zeroed in
// shared memory, or a weight of zero would make them NaN, and their tokens are listed; a row
// that sees such a token looks at those tiles' values again at its end and sets the channels
// that are not finite to NaN.
// Few rows: the keys are split over several CTAs, whose normalised parts a second kernel
// joins by their log-sum-exp.
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
constexpr int kSoftRegs = 200, kOtherRegs = 56;
static_assert(2 * kSoftRegs + 2 * kOtherRegs <= 4 * 128, "setmaxnreg.inc draws on the launch's registers");
constexpr int kPolls = 1 << 18;                // bound of a wait: a poll suspends for up to 3.7 us, so about a second
constexpr int kMaxSplits = 32;
constexpr int kPart = 132;                     // floats of a row's part: lse, 3 unused, 128 channels
constexpr float kNoRef = -3e38f;
constexpr float kRaise = 20.f;
constexpr int kStages = 2;                     // of K and of V

constexpr uint32_t kOffQ = 0;                  // two tiles
constexpr uint32_t kOffK = 2 * kOperand;
constexpr uint32_t kOffV = kOffK + kStages * kOperand;
constexpr uint32_t kOffOut = kOffV + kStages * kOperand;   // 2 KB for each softmax warp
constexpr uint32_t kOffInfo = kOffOut + 8 * 2048;

constexpr int kItems = 4;                      // ring of items
constexpr int kLists = 8;                      // ring of passes

enum { kKFull = 0, kKEmpty = kKFull + kStages, kVLand = kKEmpty + kStages, kVFull = kVLand + kStages,
       kVEmpty = kVFull + kStages, kQFull = kVEmpty + kStages, kQEmpty = kQFull + 2, kSFull = kQEmpty + 2, kPFull = kSFull + 2,
       kOFull = kPFull + 2, kDrain = kOFull + 2, kCancel, kItem, kFree = kItem + kItems, kBars = kFree + kItems };

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
  uint32_t list[kLists][4];                    // of a pass that is seen in part: tokens with values that are not finite
  uint32_t tmem;
  int abort;
  int steps;                                   // items looked at so far
  int given;                                   // items published so far
  int taken;                                   // an item taken on but not published yet, else -1
  int next[8];                                 // softmax warps, at their end: the item whose rows would have come next
};
constexpr uint32_t kSmem = kOffInfo + sizeof(Shared) + 1024;

struct PromptArgs {
  PromptCall c;
  int Hq, Hkv, G, n_split, q_blocks;
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
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Item x of the grid; false where it has no rows (the whole warp calls this).
__device__ __forceinline__ bool find_work(const PromptArgs& a, int x, Work& w) {
  // blocks of a sequence from its last (most keys) to its first
  w.split = x % a.n_split;
  x /= a.n_split;
  w.h = x % a.Hkv;
  x /= a.Hkv;
  w.s = x % a.c.n_seqs;
  const int blk = a.q_blocks - 1 - x / a.c.n_seqs;
  w.c0 = a.c.cu_q[w.s];
  w.m = a.c.cu_q[w.s + 1] - w.c0;
  w.k0 = a.c.cu_k[w.s];
  w.n = a.c.cu_k[w.s + 1] - w.k0;
  if (w.m < 0 || w.m > a.c.max_q || w.n < 0 || w.n > a.c.max_k || w.c0 < 0 || (long long)w.c0 + w.m > a.c.q_rows || w.k0 < 0 ||
      (long long)w.k0 + w.n > a.c.kv_rows) {
    if ((threadIdx.x & 31) == 0 && blk == 0 && w.split == 0 && w.h == 0) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return false;
  }
  w.row0 = blk * 2 * kRows;
  if ((long long)w.row0 >= (long long)w.m * a.G) return false;
  w.pos0 = w.n - w.m;
  const int p_lo = w.pos0 + w.row0 / a.G, p_hi = w.pos0 + min((w.row0 + 2 * kRows) / a.G, w.m) - 1;
  w.low = a.c.window ? max(p_lo - a.c.window + 1, 0) : 0;
  const int end = max(p_hi + 1, 0);
  w.first = p_lo;
  w.keys = end;
  w.sinks = a.c.window ? a.c.n_sink : 0;
  w.w0 = min(w.low, end) / kKeys;
  w.ns = min((min(w.sinks, end) + kKeys - 1) / kKeys, w.w0);
  const int total = w.ns + (end + kKeys - 1) / kKeys - w.w0;
  const int per = (total + a.n_split - 1) / a.n_split;
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

// The loads of an item: false where a wait ran out.  g, keyed: passes (of K and of V) and
// items with keys loaded so far.
__device__ __forceinline__ bool load_item(const PromptArgs& a, const Maps& maps, const Work& w, bool withhold, uint8_t* sm,
                                          Shared* sh, const Waiter& wait, int (&g)[2], int (&keyed)[2]) {
  const int lane = threadIdx.x & 31, tokens = kRows / a.G, h = w.h, k0 = w.k0, q0 = w.c0 + w.row0 / a.G;
  const uint32_t base = smem_u32(sm);
  auto ready = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(sh->bars + bar, parity)) != 0; };
  for (int tile = 0; tile < 2; ++tile) {
    if (keyed[tile] && !ready(kQEmpty + tile, (keyed[tile] - 1) & 1)) return false;
    if (lane == 0) {
      uint64_t* bar = sh->bars + kQFull + tile;
      mbar_expect_tx(bar, kOperand);
      for (int half = 0; half < 2; ++half)
        load_box(base + kOffQ + tile * kOperand + half * (kOperand / 2), maps.q, 64 * half, h * a.G, q0 + tile * tokens, bar);
    }
    ++keyed[tile];
  }
  for (int i = w.i0; i < w.i1; ++i) {
    const int row = k0 + w.tile(i) * kKeys;
    for (int kv = 0; kv < 2; ++kv) {
      const int stage = g[kv] % kStages, use = g[kv] / kStages;
      if (use && !ready((kv ? kVEmpty : kKEmpty) + stage, (use - 1) & 1)) return false;
      if (kv && withhold && i + 1 == w.i1) return false;
      if (lane == 0) {
        uint64_t* bar = sh->bars + (kv ? kVLand : kKFull) + stage;
        mbar_expect_tx(bar, kOperand);
        for (int half = 0; half < 2; ++half)
          load_box(base + (kv ? kOffV : kOffK) + stage * kOperand + half * (kOperand / 2), kv ? maps.v : maps.k, 64 * half, h,
                   row, bar);
      }
      ++g[kv];
    }
  }
  __syncwarp();
  return true;
}

__device__ __forceinline__ void load_tiles(const PromptArgs& a, const Maps& maps, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const int lane = threadIdx.x & 31;
  int g[2] = {0, 0}, keyed[2] = {0, 0};
  for (int item = 0;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) break;
    const Work& w = sh->work[slot];
    if (w.state == kStop) break;
    if (w.state == kKeyed &&
        !load_item(a, maps, w, a.stall && blockIdx.x == 0 && item == 0, sm, sh, wait, g, keyed))
      break;
    if (lane == 0) arrive(sh->bars + kFree + slot);
    __syncwarp();
  }
  // whatever happened to those who wait for them: no load may land after the CTA has ended
  for (int i = 0; i < 2; ++i)
    if (keyed[i]) mbar_wait(sh->bars + kQFull + i, (keyed[i] - 1) & 1, kPolls);
  for (int kv = 0; kv < 2; ++kv)
    for (int n = max(g[kv] - kStages, 0); n < g[kv]; ++n)
      mbar_wait(sh->bars + (kv ? kVLand : kKFull) + n % kStages, (n / kStages) & 1, kPolls);
}

// ---- values of tiles seen in part (four warps, a thread to a token) ----------------

__device__ __forceinline__ void look_through(const PromptArgs& a, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const int tid = threadIdx.x & 127, lane = threadIdx.x & 31;
  int g = 0;
  for (int item = 0;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) return;
    const Work& w = sh->work[slot];
    if (w.state == kStop) return;
    if (w.state == kKeyed) {
      for (int i = w.i0; i < w.i1; ++i, ++g) {
        const int stage = g % kStages;
        if (!__all_sync(0xffffffffu, wait(sh->bars + kVLand + stage, (g / kStages) & 1))) return;
        if (in_part(a, w, w.tile(i) * kKeys)) {
          uint8_t* row = sm + kOffV + stage * kOperand + tid * 128;
          uint32_t m = 0;
#pragma unroll
          for (int c = 0; c < 16; ++c) {       // the swizzle: eight lanes read eight different banks
            const uint4 x = *reinterpret_cast<const uint4*>(row + (c >> 3) * (kOperand / 2) + (((c ^ tid) & 7) << 4));
            m = __vmaxu2(__vmaxu2(__vmaxu2(m, x.x & 0x7FFF7FFFu), __vmaxu2(x.y & 0x7FFF7FFFu, x.z & 0x7FFF7FFFu)),
                         x.w & 0x7FFF7FFFu);
          }
          const bool bad = (m & 0xFFFFu) >= 0x7F80u || (m >> 16) >= 0x7F80u;
          const uint32_t listed = __ballot_sync(0xffffffffu, bad);
          if (lane == 0) sh->list[g & (kLists - 1)][tid >> 5] = listed;
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
          fence_async();
        }
        __syncwarp();
        if (lane == 0) arrive(sh->bars + kVFull + stage);
      }
    }
    if (lane == 0) arrive(sh->bars + kFree + slot);
    __syncwarp();
  }
}

// ---- walker (one warp) -------------------------------------------------------------

// The items: this CTA's own, then those of CTAs that have not been launched yet, asked of
// the hardware's scheduler one ahead.
__device__ __forceinline__ void walk(const PromptArgs& a, Shared* sh, const Waiter& wait) {
  const int lane = threadIdx.x & 31;
  auto ready = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(sh->bars + bar, parity)) != 0; };
  auto publish = [&](const Work& w, int item) -> bool {
    const int slot = item & (kItems - 1);
    if (item >= kItems && !ready(kFree + slot, (item / kItems - 1) & 1)) return false;
    if (lane == 0) {
      sh->work[slot] = w;
      sh->given = item + 1;
      sh->taken = -1;
      arrive(sh->bars + kItem + slot);
    }
    __syncwarp();
    return true;
  };
  int x = blockIdx.x, items = 0;
  bool ok = true;
  for (int asked = 0;; ++asked) {
    if (lane == 0) {
      fence_async();
      mbar_expect_tx(sh->bars + kCancel, 16);
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
              smem_u32(&sh->cancel)),
          "r"(smem_u32(sh->bars + kCancel))
          : "memory");
    }
    if (lane == 0) *reinterpret_cast<volatile int*>(&sh->steps) = asked + 1;
    __syncwarp();
    Work w;
    if (find_work(a, x, w)) ok = publish(w, items++);
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
    if (lane == 0) sh->taken = got ? x : -1;
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
// same instruction cache, and a short loop stays in it.
__device__ __forceinline__ void issue_products(uint32_t tmem, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const uint32_t base = smem_u32(sm);
  const uint64_t q0 = desc(base + kOffQ, 16), k0 = desc(base + kOffK, 16), v0 = desc(base + kOffV, kOperand / 2);
  auto ready = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(sh->bars + bar, parity)) != 0; };
  auto scores = [&](int tile, int stage, bool last) {
    if (elect_one()) {
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
      arrive(sh->bars + kSFull + tile);        // a release after this warp saw the lists so far
      if (tile == 1) commit(sh->bars + kKEmpty + stage);
      if (last) commit(sh->bars + kQEmpty + tile);
    }
    __syncwarp();
  };
  int g = 0, keyed = 0;                        // passes and items with keys so far
  for (int item = 0;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) return;
    const int state = sh->work[slot].state, passes = sh->work[slot].i1 - sh->work[slot].i0;
    if (state == kStop) return;
    if (state == kKeyed) {
      if (!ready(kKFull + g % kStages, (g / kStages) & 1)) return;
#pragma unroll 1
      for (int tile = 0; tile < 2; ++tile) {
        if (!ready(kQFull + tile, keyed & 1)) return;
        fence_after();
        scores(tile, g % kStages, passes == 1);
      }
      for (int it = 0; it < passes; ++it, ++g) {
        const int stage = g % kStages, next = (g + 1) % kStages;
        const bool last = it + 1 == passes;
        // V, and the K of the next scores, long since there: looked at before P is due
        if (!ready(kVFull + stage, (g / kStages) & 1)) return;
        if (!last && !ready(kKFull + next, ((g + 1) / kStages) & 1)) return;
#pragma unroll 1
        for (int tile = 0; tile < 2; ++tile) {
          if (!ready(kPFull + tile, g & 1)) return;
          fence_after();
          if (elect_one()) {
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
            if (tile == 1) commit(sh->bars + kVEmpty + stage);
            if (last) {
              arrive(sh->bars + kOFull + tile);   // a release after this warp saw the last list
              commit(sh->bars + kOFull + tile);
            }
          }
          __syncwarp();
          if (!last) scores(tile, next, it + 2 == passes);
        }
      }
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
    token = row >> (__ffs(a.G) - 1);           // G: 1, 2, 4 or 8
    hq = w.h * a.G + (row & (a.G - 1));
    live = token < w.m;
    qrow = ((size_t)w.c0 + token) * a.Hq + hq;
  }
};

struct RowOut {
  float M = kNoRef, l = 0.f;
  bool poison = false;                         // sees a listed token
};

// The keys from t0 on that row i of the block sees.
__device__ __forceinline__ void sees(const PromptArgs& a, const Work& w, int i, int t0, uint32_t (&see)[4]) {
  const int pos = w.pos0 + Row(a, w, i).token;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t m = below(pos + 1 - t0, 32 * q);
    if (a.c.window) m &= ~below(pos + 1 - a.c.window - t0, 32 * q) | below(w.sinks - t0, 32 * q);
    see[q] = m;
  }
}
// Whether it sees a listed token of pass g (known once V is there).
__device__ __forceinline__ bool poisoned(const PromptArgs& a, const Work& w, const Shared* sh, int i, int t0, int g) {
  uint32_t see[4];
  sees(a, w, i, t0, see);
  const uint32_t* list = sh->list[g & (kLists - 1)];
  return ((list[0] & see[0]) | (list[1] & see[1]) | (list[2] & see[2]) | (list[3] & see[3])) != 0;
}

// The passes of an item, up to its last weights.  g: the pass, counted over the CTA's
// items; left at the last one.
__device__ __forceinline__ bool softmax_rows(const PromptArgs& a, const Work& w, uint32_t trow, int tile, Shared* sh,
                                             const Waiter& wait, int& g, RowOut& ro) {
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
    if (check >= 0) ro.poison |= poisoned(a, w, sh, i0, check, g - 1);
    const bool part = in_part(a, w, t0);
    check = part ? t0 : -1;
    float c = cs;
    float v[kKeys];
#pragma unroll
    for (int q = 0; q < 4; ++q) ld32(ts + 32 * q, v + 32 * q);
#pragma unroll
    for (int q = 0; q < 4; ++q) settle(v + 32 * q);
    if (minus) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) v[i] = -v[i];
    }
    if (part) {
      uint32_t see[4];
      sees(a, w, i0, t0, see);
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (!((see[i >> 5] >> (i & 31)) & 1)) v[i] = -INFINITY;
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
    if ((threadIdx.x & 31) == 0) arrive(sh->bars + kPFull + tile);
    if (it + 1 == passes) return true;
  }
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

// A row's result: normalised to the output, or as a part of a split.  `stage`: 2 KB of
// shared memory for 32 channels of the warp's 32 rows, from which they are written 64 bytes
// at a time.
__device__ __forceinline__ void write_row(const PromptArgs& a, const Work& w, uint32_t to, uint8_t* stage, int row0, bool any,
                                          bool ok, const RowOut& ro) {
  const int lane = threadIdx.x & 31;
  const Row row(a, w, row0 + lane);
  const float nan = __uint_as_float(0x7FC00000u);
  const bool empty = ok && ro.l == 0.f;
  const float f = !ok ? nan : (empty ? 0.f : 1.f / ro.l);
  const float lse = !ok ? nan : lse_of(ro.M, ro.l);
  float* part = static_cast<float*>(a.c.ws) + ((((size_t)w.s * a.c.max_q + row.token) * a.Hq + row.hq) * a.n_split + w.split) * kPart;
  // where this lane's 16 bytes of the warp's rows 8 i + lane / 4 go
  uint4* dst[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Row r(a, w, row0 + 8 * i + (lane >> 2));
    dst[i] = r.live ? static_cast<uint4*>(a.c.out) + r.qrow * 16 + (lane & 3) : nullptr;
  }
  const bool read = any && ok;                 // the same for the whole warp
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float o[32];
    if (read) {
      ld32(to + 32 * q, o);
      settle(o);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = empty ? 0.f : o[i] * f;
    if (ro.poison && row.live && ok) {
      const uint32_t bits = spoiled(a, w, row0 + lane, q);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if ((bits >> i) & 1) o[i] = nan;
    }
    if (a.n_split > 1) {
      if (row.live) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(part + 4 + 32 * q + 4 * i) =
              make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = pack_bf16(o[8 * i + 2 * e], o[8 * i + 2 * e + 1]);
        // 16-byte chunk i of row r at i ^ (r / 2 % 4): no bank conflicts either way
        *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {            // eight rows per step, four lanes each
        const int r = 8 * i + (lane >> 2);
        if (dst[i]) dst[i][4 * q] = *reinterpret_cast<const uint4*>(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
      }
    }
  }
  if (row.live) {
    if (a.n_split > 1)
      part[0] = lse;
    else if (a.c.lse)
      a.c.lse[row.qrow] = lse;
  }
}

// Rows of items that a CTA took on and did not get to before it gave up: not a number (in a
// split, the row's part: the join would read what the workspace held before).  first: the
// first item whose rows this warp has not written.
__device__ __forceinline__ void abandon(const PromptArgs& a, const Shared* sh, int first) {
  const int i = threadIdx.x, given = sh->given;   // this thread's row of a block
  const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll 1
  for (int item = first; item <= given; ++item) {
    Work w;
    if (item < given)
      w = sh->work[item & (kItems - 1)];
    else if (sh->taken < 0 || !find_work(a, sh->taken, w))
      return;
    if (w.state == kStop) return;
    const Row row(a, w, i);
    if (!row.live) continue;
    if (a.n_split > 1) {
      static_cast<float*>(a.c.ws)[((((size_t)w.s * a.c.max_q + row.token) * a.Hq + row.hq) * a.n_split + w.split) * kPart] = nan;
    } else {
      uint4* out = static_cast<uint4*>(a.c.out) + row.qrow * 16;
#pragma unroll 1
      for (int c = 0; c < 16; ++c) out[c] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
      if (a.c.lse) a.c.lse[row.qrow] = nan;
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
      mbar_init(sh->bars + kKFull + i, 1);
      mbar_init(sh->bars + kKEmpty + i, 1);
      mbar_init(sh->bars + kVLand + i, 1);
      mbar_init(sh->bars + kVFull + i, 4);
      mbar_init(sh->bars + kVEmpty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh->bars + kQFull + i, 1);
      mbar_init(sh->bars + kQEmpty + i, 1);
      mbar_init(sh->bars + kSFull + i, 2);
      mbar_init(sh->bars + kPFull + i, 4);
      mbar_init(sh->bars + kOFull + i, 2);
    }
    mbar_init(sh->bars + kDrain, 1);
    mbar_init(sh->bars + kCancel, 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(sh->bars + kItem + i, 1);
      mbar_init(sh->bars + kFree + i, 2 * kRows + 6);   // softmax threads, four looking warps, loader, issuer
    }
    mbar_fence_init();
    sh->abort = 0;
    sh->steps = 0;
    sh->given = 0;
    sh->taken = blockIdx.x;
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
    const int tile = warp >> 2;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int m0 = 32 * (warp & 3);            // this warp's rows of the tile
    int g = 0, keyed = 0, item = 0;
    for (;; ++item) {
      const int slot = item & (kItems - 1);
      if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) break;
      const Work& w = sh->work[slot];
      if (w.state == kStop) break;
      RowOut ro;
      bool ok = true;
      if (w.state == kKeyed) {
        ok = softmax_rows(a, w, trow, tile, sh, wait, g, ro);
        if (ok) ok = __all_sync(0xffffffffu, wait(sh->bars + kOFull + tile, keyed & 1)) != 0;
        fence_after();
        const int t0 = w.tile(w.i1 - 1) * kKeys;
        if (ok && in_part(a, w, t0)) ro.poison |= poisoned(a, w, sh, tile * kRows + (threadIdx.x & 127), t0, g);
        ++g;
        ++keyed;
      }
      write_row(a, w, trow + 256 + 128 * tile, sm + kOffOut + warp * 2048, tile * kRows + m0, w.state == kKeyed, ok, ro);
      arrive(sh->bars + kFree + slot);
      if (!ok) {
        ++item;
        break;
      }
    }
    if ((threadIdx.x & 31) == 0) sh->next[warp] = item;   // kept there: held in a register to the end it costs spills
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < 12) look_through(a, sm, sh, wait);
    if (warp == 12) issue_products(__shfl_sync(0xffffffffu, tmem, 0), sm, sh, wait);
    if (warp == 13) walk(a, sh, wait);
    if (warp == 14) load_tiles(a, {&mq, &mk, &mv}, sm, sh, wait);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp < 8 && sh->abort) abandon(a, sh, sh->next[warp]);
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
  const int c0 = a.c.cu_q[s], m = a.c.cu_q[s + 1] - c0, k0 = a.c.cu_k[s], n = a.c.cu_k[s + 1] - k0;
  if (m > a.c.max_q || i >= m || n < 0 || n > a.c.max_k || c0 < 0 || (long long)c0 + m > a.c.q_rows || k0 < 0 ||
      (long long)k0 + n > a.c.kv_rows)
    return;
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

long long q_blocks(const Pool& p, int max_q) { return ((long long)max_q * p.G + 2 * kRows - 1) / (2 * kRows); }

// Splits of the keys: where the blocks of rows fill less than half of the SMs, as many as
// fit in one wave, of at least four tiles each.
int splits(const Pool& p, int n_seqs, int max_q, long long max_k, int window, int n_sink) {
  long long keys = max_k;
  if (window) keys = std::min(keys, (long long)window + n_sink + std::min<long long>(max_q, 2 * kRows / p.G) + 2 * kKeys);
  const long long tiles = (keys + kKeys - 1) / kKeys, blocks = q_blocks(p, max_q) * n_seqs * p.cfg.num_kv_heads;
  if (blocks == 0) return 1;
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
  if (c.max_q == 0) return cudaSuccess;
  PromptArgs a{c, p.cfg.num_q_heads, p.cfg.num_kv_heads, p.G, splits(p, c.n_seqs, c.max_q, c.max_k, c.window, c.n_sink),
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
