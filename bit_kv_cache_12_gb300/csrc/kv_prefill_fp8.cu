// Prompt attention over the 8-bit cache on the tcgen05 tensor cores.
//
// A row is a (query token, query head of the KV head) pair, so the G heads that
// share a KV head share its tiles: a block of 256 rows holds 256 / G tokens.
// Per row, with base-2 logits  x_j = |scale| log2(e) 2^eK (q . k_j) + eV  (codes
// k, v of exponents eK, eV; q carries scale's sign):
//   w_j = 2^(x_j - M),   out = sum_j w_j v_j / sum_j w_j 2^-eV.
// Operands are fp16: e4m3 codes times a power of two convert exactly (the 16
// token blocks of a 128-token tile are taken together while their exponents lie
// within 14 of one another, else in several passes); q is scaled per row by a
// power of two (largest element in [2^14, 2^15): exact for bf16's 8 bits down
// to 2^-32 of it); the weights are rounded to fp16 relative to their own size,
// between 2^-31 of the largest and 2^15, M lagging behind the running maximum
// so that the accumulator is rescaled only when a weight would pass 2^15.
//
// Bound: the tensor cores (4 * 128 operations per row and key).  One CTA per SM: two
// tiles of 128 rows take turns, one in the tensor cores while the other is in the
// softmax.  8192 tokens (32 query heads, 8 KV heads): 409 us, 1.35 PFLOP/s, 0.68 of
// the bf16 rate of a large library product; behind 32,768 cached tokens 1.56 PFLOP/s
// (0.79).  A key tile takes 3,340 clocks, its products 2,048: a tile's own chain
// (weights seen by the issuer, O += P V, S, scores seen, softmax) fills 3,310 of them,
// and taking exponentials, maximum or conversions out changes the time by 2% at most.
// An item's end costs 7 us more (last product, next q, rows written, first scores).
//   warps 0-3, 4-7   softmax of a tile: a thread owns a row; S is read from
//                    tensor memory, the weights go back over it as fp16; then
//                    the next item's q and this item's rows
//   warps 8-11       converters: codes from global memory to registers a tile
//                    ahead, fp16 in the swizzled operand layout to shared memory
//                    (two stages each of K and V)
//   warp 12          issues the products: S = Q K^T from shared memory, O += P V
//                    with P from tensor memory and V token-major as it is stored
//   warp 13          (14, 15 idle) walks the items and their key tiles ahead of
//                    the converters: page ids, exponents, block addresses into a
//                    ring of records
// Tensor memory: S0, S1 (P over them), O0, O1, 128 columns each.
// Hidden keys: a tile that some row sees only in part is masked by select after
// the product (a NaN in a hidden K row never enters), its V rows that hold NaN
// are zeroed and listed, and a row that sees one of those becomes NaN as a whole
// (the append stores a row with a NaN as NaN in every channel).
// Few rows: the keys are split over several CTAs, whose normalised parts a
// second kernel joins by their log-sum-exp.
#include <algorithm>

#include "kv_fp8.h"
#include "kv_tc.cuh"

namespace kvint2 {

namespace {

constexpr int kRows = 128;                     // rows of a tile (M of a product)
constexpr int kKeys = 128;                     // keys of a tile
constexpr int kBlocks = kKeys / kTile;
constexpr int kThreads = 16 * 32;              // four warpgroups
// registers per thread of the softmax, converter and issuer warpgroups: they
// share the launch's 128 each
constexpr int kSoftRegs = 184, kConvRegs = 96, kIssueRegs = 48;
static_assert(2 * kSoftRegs + kConvRegs + kIssueRegs <= 4 * 128, "setmaxnreg.inc draws on the launch's registers");
constexpr int kPolls = 1 << 18;                // bound of a wait: a poll suspends for up to 3.7 us, so about a second
constexpr int kMaxSplits = 32;
constexpr float kNoRef = -3e38f;
constexpr float kRaise = 15.f, kHead = 7.f;

constexpr uint32_t kOffQ = 0;                  // two tiles
constexpr uint32_t kOffK = 2 * kOperand;       // two stages
constexpr uint32_t kOffV = 4 * kOperand;       // two stages
constexpr uint32_t kOffOut = 6 * kOperand;     // 2 KB for each softmax warp
constexpr uint32_t kOffInfo = kOffOut + 8 * 2048;

// A pass over a key tile: what the walker tells the other warps; a ring of eight.
struct Pass {
  int t0;                                      // first key
  uint32_t blocks;                             // 16-token blocks present in this pass
  float fk, ev;                                // 2^eK, eV of the operands
  int last;                                    // the item's last pass
  int partial;                                 // some row sees the tile only in part
  int keys;                                    // keys from here on are hidden from every row
  int stop;                                    // not a pass: no item follows
  uint32_t nan[4];                             // its V rows that hold NaN, zeroed (by the converters)
  int tile[kBlocks];                           // stored tile of each block (0 for an absent one)
  uint32_t mulk[kBlocks], mulv[kBlocks];       // fp16x2 2^(e - eK), 2^(e - eV)
};
constexpr int kRing = 8;

constexpr int kItems = 4;                      // ring of items

enum { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPFull = 10, kOFull = 12, kQFull = 14, kDrain = 16,
       kCancel = 17, kItem = 18, kFree = kItem + kItems, kPass = kFree + kItems, kBars = kPass + kRing };

// An item: a block of rows and the key tiles they see.
enum { kKeyed = 0, kNoKeys = 1, kStop = 2, kStart = 3 };   // rows with keys, rows that see none, no item; before the first
struct Work {
  int state;
  int s, h, c0, m, n, row0, split;             // sequence, KV head, first q row, queries, keys, first row of the block
  int pos0;                                    // position of the sequence's query 0
  int first, keys;                             // position of the first row; keys from here on are hidden from every row
  int low, sinks, ns, w0, i0, i1;              // tile list: the first ns tiles, then from w0; this split's part of it
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : i - ns + w0; }
};

struct Shared {
  Pass pass[kRing];
  uint4 cancel;                                // what the scheduler answered
  Work work[kItems];
  uint64_t bars[kBars];
  uint32_t tmem;
  int abort;
  int converted;                               // passes whose K is in shared memory
  int steps;                                   // items looked at so far
  int given;                                   // items published so far
  int taken[2];                                // blocks taken on but not published: the one at hand, and (when that one
                                               // never will be) the one that the scheduler had been asked for; else -1
  int next[8];                                 // softmax warps, at their end: the item whose rows would have come next
};
constexpr uint32_t kSmem = kOffInfo + sizeof(Shared) + 1024;

struct PrefillFp8Args {
  Fp8Layer L;
  AttnCall c;
  const int32_t* cu;
  int n_seqs, max_q, Hq, G, n_split, q_blocks;
  int* err;
  int polls;
  int stall;                                   // test hook: CTA 0's walker withholds its first item's last pass (1), or
                                               // its issuer does nothing (2; asked in the converters' loop it costs 2%)
};

// ---- tcgen05 ----------------------------------------------------------------

// kind::f16, fp32 accumulator, fp16 operands, M = N = 128; bit 16: B is MN-major
constexpr uint32_t kIdescQK = (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);

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
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) {   // codes in bytes 0, 1 -> fp16x2
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Whether a sequence's rows [c0, c1) are ones, as many as it may have.  (Their difference is taken
// when they are known to be in order: others could pass 32 bits.)
__device__ __forceinline__ bool rows_in_range(const PrefillFp8Args& a, int c0, int c1) {
  return c0 >= 0 && c1 >= c0 && c1 - c0 <= a.max_q;
}

// Item x of the grid; false where it has no rows (the whole warp calls this).
__device__ __forceinline__ bool find_work(const PrefillFp8Args& a, int x, Work& w) {
  // blocks of a sequence from its last (most keys) to its first
  w.split = x % a.n_split;
  x /= a.n_split;
  w.h = x % a.L.Hkv;
  x /= a.L.Hkv;
  w.s = x % a.n_seqs;
  const int blk = a.q_blocks - 1 - x / a.n_seqs;
  w.c0 = a.cu[w.s];
  const int c1 = a.cu[w.s + 1];
  w.n = a.c.seq_len[w.s];
  const bool first = (threadIdx.x & 31) == 0 && blk == 0 && w.split == 0 && w.h == 0;
  if (!rows_in_range(a, w.c0, c1)) {
    if (first) flag_error(a.err, KV_DEVERR_SEQ_RANGE);
    return false;
  }
  w.m = c1 - w.c0;
  if (w.n < 0 || w.n > a.c.max_len) {
    if (first) flag_error(a.err, KV_DEVERR_LENGTH);
    w.n = min(max(w.n, 0), a.c.max_len);
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

// ---- converters (128 threads) -------------------------------------------------

__device__ __forceinline__ void store_run(uint8_t* operand, int token, int run, const uint4& w, uint32_t mul) {
  uint32_t f[8];
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  const __half2 m = u32_as_h2(mul);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = h2_as_u32(__hmul2(u32_as_h2(cvt_lo(x[i])), m));
    f[2 * i + 1] = h2_as_u32(__hmul2(u32_as_h2(cvt_hi(x[i])), m));
  }
  uint8_t* row = operand + (run >> 2) * (kOperand / 2) + token * 128;
  const int c = 2 * (run & 3), sw = token & 7;
  *reinterpret_cast<uint4*>(row + ((c ^ sw) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<uint4*>(row + (((c + 1) ^ sw) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
}

// 2^d, d <= 0 (0 below fp16's range), in both halves
__device__ __forceinline__ uint32_t half_pow2(int d) {
  return h2_as_u32(__float2half2_rn(pow2i(max(min(d, 0), -126))));
}

__device__ __forceinline__ bool has_nan(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }

// K and V of every pass.
__device__ __forceinline__ void convert_tiles(const PrefillFp8Args& a, uint8_t* sm, Shared* sh, const Waiter& wait) {
  const int tid = threadIdx.x & 127;
  // this thread's piece of a stored block of K and of V: token and run of 16
  // channels, chosen so that eight lanes store to eight different banks
  const int ktok = 8 * (tid >> 6) + ((tid >> 2) & 7), krun = 4 * ((tid >> 5) & 1) + (tid & 3);
  const int vtok = 8 * (tid >> 6) + (tid & 7), vrun = (tid >> 3) & 7;
  const uint8_t* ksrc = a.L.codes + tid * 16;
  const uint8_t* vsrc = a.L.codes + 2048 + ((tid & 1) + 2 * (tid >> 6)) * 512 + vrun * 64 + ((tid & 7) >> 1) * 16;
  uint4 k[kBlocks], v[kBlocks];                // a pass ahead
  auto load = [&](uint4 (&x)[kBlocks], const uint8_t* src, const Pass& p) {
#pragma unroll
    for (int u = 0; u < kBlocks; u += 4) {
      const int4 t = *reinterpret_cast<const int4*>(p.tile + u);
      x[u] = ld_stream_v4(src + (size_t)t.x * kFp8TileBytes);
      x[u + 1] = ld_stream_v4(src + (size_t)t.y * kFp8TileBytes);
      x[u + 2] = ld_stream_v4(src + (size_t)t.z * kFp8TileBytes);
      x[u + 3] = ld_stream_v4(src + (size_t)t.w * kFp8TileBytes);
    }
  };
  auto ready = [&](int it) { return __all_sync(0xffffffffu, wait.handed(sh->bars + kPass + (it & (kRing - 1)), (it / kRing) & 1)); };
  if (!ready(0) || sh->pass[0].stop) return;
  load(k, ksrc, sh->pass[0]);
  load(v, vsrc, sh->pass[0]);
  for (int it = 0;; ++it) {
    const int stage = it & 1;
    const uint32_t ph = ((it >> 1) & 1) ^ 1;   // of the empty barriers: the use before this one
    Pass& p = sh->pass[it & (kRing - 1)];
    const Pass& next = sh->pass[(it + 1) & (kRing - 1)];
    const bool partial = p.partial != 0, last = p.last != 0;
    const uint32_t present = p.blocks;
    const int t0 = p.t0, keys = p.keys;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (it >= 2 && !__all_sync(0xffffffffu, wait(sh->bars + kKEmpty + stage, ph))) return;
    uint8_t* sk = sm + kOffK + stage * kOperand;
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      if (partial && !((present >> u) & 1)) k[u] = zero;
      store_run(sk, kTile * u + ktok, krun, k[u], p.mulk[u]);
    }
    fence_async();
    arrive(sh->bars + kKFull + stage);
    if (tid == 0) *reinterpret_cast<volatile int*>(&sh->converted) = it + 1;
    if (!last) {
      if (!ready(it + 1)) return;
      load(k, ksrc, next);
    }
    if (it >= 2 && !__all_sync(0xffffffffu, wait(sh->bars + kVEmpty + stage, ph))) return;
    uint8_t* sv = sm + kOffV + stage * kOperand;
    if (partial) {
#pragma unroll
      for (int u = 0; u < kBlocks; ++u) {
        const int tok = kTile * u + vtok;
        if (!((present >> u) & 1) || t0 + tok >= keys) v[u] = zero;
        if (has_nan(v[u].x) || has_nan(v[u].y) || has_nan(v[u].z) || has_nan(v[u].w)) {
          v[u] = zero;
          atomicOr(&p.nan[tok >> 5], 1u << (tok & 31));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) store_run(sv, kTile * u + vtok, vrun, v[u], p.mulv[u]);
    fence_async();
    arrive(sh->bars + kVFull + stage);
    if (last) {                                // the next item's first pass may be long in coming
      if (!ready(it + 1) || next.stop) return;
      load(k, ksrc, next);
    }
    load(v, vsrc, next);
  }
}

// ---- walker (one warp) ----------------------------------------------------------

// Whether the record of pass n may be written: pass n - 8 was last read by the
// softmax of pass n - 7, over when K of pass n - 4 has its stage.
__device__ __forceinline__ bool pass_free(Shared* sh, const Waiter& wait, int n) {
  bool ok = true;
  for (int spin = 0; n >= kRing && *reinterpret_cast<volatile int*>(&sh->converted) < n - 3; ++spin) {
    if (spin / 32 >= wait.polls || *reinterpret_cast<volatile int*>(wait.abort)) {
      ok = false;
      break;
    }
    __nanosleep(100);                          // 32 of these to a poll of a barrier
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) *reinterpret_cast<volatile int*>(wait.abort) = 1;
  return ok;
}

// The passes of an item: a tile's blocks whose exponents lie within 7 of the first one left
// make a pass.  Lane u < 8 holds block u: its stored tile (-1: absent) and
// exponents for tile i, its exponents in flight for tile i + 1, its page id in
// flight for tile i + 2; no load waits where it is issued.
__device__ __forceinline__ bool walk_item(const PrefillFp8Args& a, const Work& w, Shared* sh, const Waiter& wait, int& n) {
  const int lane = threadIdx.x & 31;
  const int tpp = a.L.P / kTile, shift = tpp >> 1;
  const int32_t* pt = a.c.pt + (size_t)w.s * a.c.max_pages;
  auto seen = [&](int i) -> bool {             // by some row; a page that none sees may have been given up
    const int j0 = (w.tile(i) * kBlocks + lane) * kTile;
    return i < w.i1 && lane < kBlocks && j0 < w.keys && !(a.c.window && j0 + kTile <= w.low && j0 >= w.sinks);
  };
  auto page_of = [&](int i) -> int { return pt[seen(i) ? (w.tile(i) * kBlocks + lane) >> shift : 0]; };
  auto stored = [&](int i, int pid) -> int {   // below 2^31: 4 KB each
    if (!seen(i)) return -1;
    if (pid < 0 || pid >= a.L.num_pages) {
      flag_error(a.err, KV_DEVERR_PAGE_ID);
      return -1;
    }
    return (pid * a.L.Hkv + w.h) * tpp + ((w.tile(i) * kBlocks + lane) & (tpp - 1));
  };
  auto exps_of = [&](int st) -> int { return *reinterpret_cast<const uint16_t*>(a.L.exps + (size_t)max(st, 0) * 2); };
  int st1 = stored(w.i0, page_of(w.i0));
  int ex1 = exps_of(st1), pid2 = page_of(w.i0 + 1);
  for (int i = w.i0; i < w.i1; ++i) {
    const int st = st1, ex = ex1, t0 = w.tile(i) * kKeys;
    st1 = stored(i + 1, pid2);
    ex1 = exps_of(st1);
    pid2 = page_of(i + 2);
    uint32_t left = __ballot_sync(0xffffffffu, st >= 0);
    const int ek = (int8_t)(ex & 0xFF), ev = (int8_t)(ex >> 8);
    do {
      uint32_t now = 0;
      int mk = 0, mv = 0;
      if (left) {
        const int first = __shfl_sync(0xffffffffu, ex, __ffs(left) - 1);
        const bool in =
            ((left >> lane) & 1) && abs(ek - (int8_t)(first & 0xFF)) <= 7 && abs(ev - (int8_t)(first >> 8)) <= 7;
        now = __ballot_sync(0xffffffffu, in);
        mk = __reduce_max_sync(0xffffffffu, in ? ek : -1000);
        mv = __reduce_max_sync(0xffffffffu, in ? ev : -1000);
        left &= ~now;
      }
      if (!pass_free(sh, wait, n)) return false;
      Pass& p = sh->pass[n & (kRing - 1)];
      if (lane < kBlocks) {
        const bool in = (now >> lane) & 1;
        p.tile[lane] = in ? st : 0;
        p.mulk[lane] = half_pow2(ek - mk);
        p.mulv[lane] = half_pow2(ev - mv);
        if (lane < 4) p.nan[lane] = 0;
      }
      const bool last = i + 1 == w.i1 && !left;
      if (lane == 0) {
        p.t0 = t0;
        p.blocks = now;
        p.fk = pow2i(max(min(mk, 127), -126));
        p.ev = (float)mv;
        p.last = last;
        p.keys = w.keys;
        p.stop = 0;
        p.partial = now != 0xFFu || t0 + kKeys - 1 > w.first ||
                    (a.c.window && t0 < w.keys - a.c.window && t0 + kKeys > w.sinks);
      }
      __syncwarp();
      if (a.stall == 1 && last && blockIdx.x == 0) return false;
      if (lane == 0) arrive(sh->bars + kPass + (n & (kRing - 1)));
      ++n;
    } while (left);
  }
  return true;
}

// The items: this CTA's own, then those of CTAs that have not been launched yet,
// asked of the hardware's scheduler one ahead.  So a CTA lives as long as there is
// work, the walker and the converters are at the next item's keys while the
// softmax writes the last one's rows, and blocks of unequal length even out.
__device__ __forceinline__ void walk(const PrefillFp8Args& a, Shared* sh, const Waiter& wait) {
  const int lane = threadIdx.x & 31;
  auto ready = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(sh->bars + bar, parity)) != 0; };
  auto publish = [&](const Work& w, int item) -> bool {
    const int slot = item & (kItems - 1);
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
  int x = blockIdx.x, items = 0, passes = 0;
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
    if (find_work(a, x, w)) ok = publish(w, items++) && (w.state != kKeyed || walk_item(a, w, sh, wait, passes));
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
  if (!publish(stop, items) || !pass_free(sh, wait, passes)) return;
  if (lane == 0) {
    sh->pass[passes & (kRing - 1)].stop = 1;
    arrive(sh->bars + kPass + (passes & (kRing - 1)));
  }
  __syncwarp();
}

// ---- product issuer (one warp) ----------------------------------------------------

// The whole warp runs this, in step, and one lane of it issues: addresses stay in
// uniform registers.  The loops are not unrolled: the code of the other warps
// passes through the same instruction cache, and a short loop stays in it.
__device__ __forceinline__ void issue_products(bool none, uint32_t tmem, uint8_t* sm, Shared* sh, const Waiter& wait) {
  if (none) return;
  const uint32_t base = smem_u32(sm);
  const uint64_t q0 = desc(base + kOffQ, 16), k0 = desc(base + kOffK, 16), v0 = desc(base + kOffV, kOperand / 2);
  auto ready = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(sh->bars + bar, parity)) != 0; };
  auto scores = [&](int tile, int stage) {
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
      arrive(sh->bars + kSFull + tile);        // a release after this warp saw the tile's record
      if (tile == 1) commit(sh->bars + kKEmpty + stage);
    }
    __syncwarp();
  };
  int g = 0, keyed = 0;                        // passes and items with keys so far
  for (int item = 0;; ++item) {
    const int slot = item & (kItems - 1);
    if (!__all_sync(0xffffffffu, wait.handed(sh->bars + kItem + slot, (item / kItems) & 1))) return;
    const int state = sh->work[slot].state;
    if (state == kStop) return;
    if (state == kKeyed) {
      if (!ready(kKFull + (g & 1), (g >> 1) & 1)) return;
#pragma unroll 1
      for (int tile = 0; tile < 2; ++tile) {
        if (!ready(kQFull + tile, keyed & 1)) return;
        fence_after();
        scores(tile, g & 1);
      }
      bool last = false;
      for (int it = 0; !last; ++it, ++g) {
        const int stage = g & 1;
        last = sh->pass[g & (kRing - 1)].last != 0;
        // V, and the K of the next scores, long since there: looked at before P is due
        if (!ready(kVFull + stage, (g >> 1) & 1)) return;
        if (!last && !ready(kKFull + (stage ^ 1), ((g + 1) >> 1) & 1)) return;
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
              arrive(sh->bars + kOFull + tile);   // a release after this warp saw the last V's record
              commit(sh->bars + kOFull + tile);
            }
          }
          __syncwarp();
          if (!last) scores(tile, stage ^ 1);
        }
      }
      ++keyed;
    }
    if (elect_one()) arrive(sh->bars + kFree + slot);
    __syncwarp();
  }
}

// ---- softmax (a thread owns a row) ---------------------------------------------

// Where row i of an item's block comes from and goes to.
struct Row {
  int token, hq;
  bool live;
  size_t qrow;
  __device__ __forceinline__ Row(const PrefillFp8Args& a, const Work& w, int i) {
    const int row = w.row0 + i;                // of the sequence's rows
    token = row >> (__ffs(a.G) - 1);           // G: 1, 2, 4 or 8
    hq = w.h * a.G + (row & (a.G - 1));
    live = token < w.m;
    qrow = ((size_t)w.c0 + token) * a.Hq + hq;
  }
};

struct RowOut {
  float M = kNoRef, l = 0.f;
  bool poison = false;
};

// The keys of a pass that row i of the block sees.
__device__ __forceinline__ void sees(const PrefillFp8Args& a, const Work& w, int i, const Pass& p, uint32_t (&see)[4]) {
  const int pos = w.pos0 + Row(a, w, i).token, t0 = p.t0;
  const uint32_t blocks = p.blocks;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t m = below(pos + 1 - t0, 32 * q);
    if (a.c.window) m &= ~below(pos + 1 - a.c.window - t0, 32 * q) | below(w.sinks - t0, 32 * q);
    m &= ((blocks >> (2 * q)) & 1 ? 0xFFFFu : 0u) | ((blocks >> (2 * q + 1)) & 1 ? 0xFFFF0000u : 0u);
    see[q] = m;
  }
}
// Whether it sees a key whose V row holds NaN (known once V is there).
__device__ __forceinline__ bool poisoned(const PrefillFp8Args& a, const Work& w, int i, const Pass& p) {
  if (!p.partial) return false;
  uint32_t see[4];
  sees(a, w, i, p, see);
  return ((p.nan[0] & see[0]) | (p.nan[1] & see[1]) | (p.nan[2] & see[2]) | (p.nan[3] & see[3])) != 0;
}

// The passes of an item, up to its last weights.  g: the pass, counted over the CTA's
// items; left at the last one.
__device__ __forceinline__ bool softmax_rows(const PrefillFp8Args& a, const Work& w, uint32_t trow, int tile, Shared* sh,
                                             const Waiter& wait, float cs, int& g, RowOut& ro) {
  const uint32_t ts = trow + 128 * tile, to = trow + 256 + 128 * tile;
  const int i0 = tile * kRows + (threadIdx.x & 127);
  bool check = false;                          // the pass before was partial
  bool large = false;                          // this row's reference is
  for (int it = 0;; ++it, ++g) {
    if (!__all_sync(0xffffffffu, wait(sh->bars + kSFull + tile, g & 1))) return false;
    fence_after();
    const Pass& info = sh->pass[g & (kRing - 1)];
    if (check) ro.poison |= poisoned(a, w, i0, sh->pass[(g - 1) & (kRing - 1)]);
    const bool partial = info.partial != 0, last = info.last != 0;
    check = partial;
    // above 0, so that a hidden key's -inf stays one
    float c = fmaxf(cs * info.fk, 1.17549435e-38f);
    const float ev = info.ev;
    float v[kKeys];
#pragma unroll
    for (int q = 0; q < 4; ++q) ld32(ts + 32 * q, v + 32 * q);
#pragma unroll
    for (int q = 0; q < 4; ++q) settle(v + 32 * q);
    if (partial) {
      uint32_t see[4];
      sees(a, w, i0, info, see);
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
    const float x = fmaf(max3(fmaxf(top[0], top[1]), top[2], top[3]), c, ev);
    const bool raise = x - ro.M > kRaise;      // as a difference: where M is large, M + 15 is rounded by as much as that
    float d = ev - ro.M;
    if (__any_sync(0xffffffffu, raise || large)) {
      const float n = raise ? x - kHead : ro.M;
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
      d = ev - n;
      large = large_reference(n);
      if (large) {                             // weights from the rounded logits; in here, where no usual pass comes by
        const uint64_t cc = f2(c, c), ee = f2(ev, ev), mm = f2(-n, -n);
#pragma unroll
        for (int i = 0; i < kKeys; i += 2) f2_split(f2_add(f2_fma(f2(v[i], v[i + 1]), cc, ee), mm), v[i], v[i + 1]);
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
        p[i] = pack_f16(y0, y1);
      }
      st16(ts + 16 * q, p);
    }
    float sa, sb;
    f2_split(f2_add(s0, s1), sa, sb);
    ro.l = fmaf(sa + sb, exp2f(-ev), ro.l);
    wait_st();
    fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive(sh->bars + kPFull + tile);
    if (last) return true;
  }
}

// The warp's 32 rows of q (first row m0 of the block), half a warp to a row: on their
// way to registers.
__device__ __forceinline__ void fetch_q(const PrefillFp8Args& a, const Work& w, int m0, uint4 (&x)[16]) {
  const int lane = threadIdx.x & 31, half = lane >> 4, shift = __ffs(a.G) - 1;   // G: 1, 2, 4 or 8, and rows a multiple
  const int token = (w.row0 + m0) >> shift, live = (w.m - token) << shift;
  const uint8_t* src = static_cast<const uint8_t*>(a.c.q) + (lane & 15) * 16 +
                       ((long long)(w.c0 + token) * a.Hq + w.h * a.G) * 256;
#pragma unroll
  for (int i = 0; i < 16; ++i) {               // rows 2 i and 2 i + 1
    const int r = 2 * i + half;
    x[i] = make_uint4(0, 0, 0, 0);
    if (r < live)
      x[i] = *reinterpret_cast<const uint4*>(src + (long long)((r >> shift) * a.Hq + (r & (a.G - 1))) * 256);
  }
}

// Those rows, each scaled by a power of two, as fp16 into the swizzled operand; returns
// the factor that brings a score of this thread's row back to base-2 logits (without 2^eK).
__device__ __forceinline__ float store_q(const PrefillFp8Args& a, uint8_t* operand, int m0, const uint4 (&x)[16]) {
  const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = __vmaxu2(top, w[u] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    const uint32_t t0 = __reduce_max_sync(0xffffffffu, half ? 0u : top);
    const uint32_t t1 = __reduce_max_sync(0xffffffffu, half ? top : 0u);
    if ((lane >> 1) == i) mine = (lane & 1) ? t1 : t0;   // row `lane` is row 2 (lane / 2) + lane % 2
    top = half ? t1 : t0;
    float mul = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : pow2i(min(14 - ((int)(top >> 7) - 127), 127));
    if (a.c.scale < 0.f) mul = -mul;
    uint32_t f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) f[u] = pack_f16(bf16lo(w[u]) * mul, bf16hi(w[u]) * mul);
    const int m = m0 + 2 * i + half;
    *reinterpret_cast<uint4*>(operand + (c >> 3) * (kOperand / 2) + m * 128 + (((c & 7) ^ (m & 7)) << 4)) =
        make_uint4(f[0], f[1], f[2], f[3]);
  }
  fence_async();
  const int up = min(14 - ((mine >> 7) - 127), 127);
  return fabsf(a.c.scale) * 1.4426950408889634f * pow2i(max(-up, -126));
}

// A row's result: normalised to the output, or as a part of a split.  `stage`:
// 2 KB of shared memory for 32 channels of the warp's 32 rows, from which they are
// written 64 bytes at a time.
__device__ __forceinline__ void write_row(const PrefillFp8Args& a, const Work& w, uint32_t to, uint8_t* stage, int row0,
                                          bool any, bool ok, const Row& row, const RowOut& ro) {
  const int lane = threadIdx.x & 31, token = row.token, hq = row.hq;
  const size_t qrow = row.qrow;
  const bool live = row.live;
  const float nan = __uint_as_float(0x7FC00000u);
  const bool empty = ok && !ro.poison && ro.l == 0.f;
  const float f = !ok || ro.poison ? nan : (empty ? 0.f : 1.f / ro.l);
  const float lse = !ok ? nan : lse_of(ro.M, ro.l);
  float* part = static_cast<float*>(a.c.ws) +
                (((size_t)w.s * a.max_q + token) * a.Hq + hq) * a.n_split * 132 + (size_t)w.split * 132;
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
    if (a.n_split > 1) {
      if (live) {
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
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 y = __floats2bfloat162_rn(o[8 * i + 2 * e], o[8 * i + 2 * e + 1]);
          u[e] = *reinterpret_cast<const uint32_t*>(&y);
        }
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
  if (live) {
    if (a.n_split > 1)
      part[0] = lse;
    else if (a.c.lse)
      a.c.lse[qrow] = lse;
  }
}

// Rows of items that a CTA took on and did not get to before it gave up: not a number
// (in a split, the row's part: the join would read what the workspace held before).
// first: the first item whose rows this warp has not written.
__device__ __forceinline__ void abandon(const PrefillFp8Args& a, const Shared* sh, int first) {
  const int i = threadIdx.x, given = sh->given;   // this thread's row of a block
  const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll 1
  for (int item = first; item < given + 2; ++item) {
    Work w;
    if (item < given)
      w = sh->work[item & (kItems - 1)];
    else if (sh->taken[item - given] < 0 || !find_work(a, sh->taken[item - given], w))
      continue;
    if (w.state == kStop) return;
    const Row row(a, w, i);
    if (!row.live) continue;
    if (a.n_split > 1) {
      static_cast<float*>(a.c.ws)[((((size_t)w.s * a.max_q + row.token) * a.Hq + row.hq) * a.n_split + w.split) * 132] = nan;
    } else {
      uint4* out = static_cast<uint4*>(a.c.out) + row.qrow * 16;
#pragma unroll 1
      for (int c = 0; c < 16; ++c) out[c] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
      if (a.c.lse) a.c.lse[row.qrow] = nan;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) prefill_fp8_kernel(PrefillFp8Args a) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Shared* sh = reinterpret_cast<Shared*>(sm + kOffInfo);
  const int warp = threadIdx.x >> 5;
  release_successor();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh->bars + kKFull + i, 128);
      mbar_init(sh->bars + kVFull + i, 128);
      mbar_init(sh->bars + kKEmpty + i, 1);
      mbar_init(sh->bars + kVEmpty + i, 1);
      mbar_init(sh->bars + kSFull + i, 2);
      mbar_init(sh->bars + kPFull + i, 4);
      mbar_init(sh->bars + kQFull + i, 128);
      mbar_init(sh->bars + kOFull + i, 2);
    }
    mbar_init(sh->bars + kDrain, 1);
    mbar_init(sh->bars + kCancel, 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(sh->bars + kItem + i, 1);
      mbar_init(sh->bars + kFree + i, 2 * kRows + 1);
    }
    for (int i = 0; i < kRing; ++i) mbar_init(sh->bars + kPass + i, 1);
    mbar_fence_init();
    sh->abort = 0;
    sh->converted = 0;
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
    const int tile = warp >> 2, m = threadIdx.x & 127;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int m0 = 32 * (warp & 3);            // this warp's rows of the tile
    auto given = [&](int item) {
      return __all_sync(0xffffffffu, wait.handed(sh->bars + kItem + (item & (kItems - 1)), (item / kItems) & 1)) != 0;
    };
    bool ok = true;
    int g = 0, keyed = 0, state = kStart;
    float cs = 0.f;
    int item = -1;
    for (; state != kStop; ++item) {
      const Work& w = sh->work[item & (kItems - 1)];
      RowOut ro;
      if (state == kKeyed) ok = softmax_rows(a, w, trow, tile, sh, wait, cs, g, ro);
      // The next item's q takes this one's place, whose last scores are read, while
      // the last product runs; its first scores form while this item's rows are written.
      const Work& next = sh->work[(item + 1) & (kItems - 1)];
      int next_state = kStop;
      uint4 x[16];
      if (ok && given(item + 1)) {
        next_state = next.state;
        if (next_state == kKeyed) {            // one line each of the warp's 32 rows
          const Row r(a, next, tile * kRows + m);
          if (r.live) {
            const uint8_t* line = static_cast<const uint8_t*>(a.c.q) + r.qrow * 256;
            prefetch_l2(line);
            prefetch_l2(line + 128);
          }
        }
      }
      if (next_state == kKeyed) {
        fetch_q(a, next, tile * kRows + m0, x);
        cs = store_q(a, sm + kOffQ + tile * kOperand, m0, x);
        arrive(sh->bars + kQFull + tile);
      }
      if (ok && state == kKeyed) {
        ok = __all_sync(0xffffffffu, wait(sh->bars + kOFull + tile, keyed & 1)) != 0;
        fence_after();
        ro.poison |= poisoned(a, w, tile * kRows + m, sh->pass[g & (kRing - 1)]);
        ++g;
        ++keyed;
      }
      if (state != kStart) {
        write_row(a, w, trow + 256 + 128 * tile, sm + kOffOut + warp * 2048, tile * kRows + m0, state == kKeyed, ok,
                  Row(a, w, tile * kRows + m), ro);
        arrive(sh->bars + kFree + (item & (kItems - 1)));
      }
      state = ok ? next_state : kStop;
    }
    if ((threadIdx.x & 31) == 0) sh->next[warp] = item;   // kept there: held in a register to the end it costs spills
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    convert_tiles(a, sm, sh, wait);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 13) walk(a, sh, wait);
    if (warp == 12) issue_products(a.stall == 2 && blockIdx.x == 0, __shfl_sync(0xffffffffu, tmem, 0), sm, sh, wait);
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
__global__ void __launch_bounds__(256) prefill_join_kernel(PrefillFp8Args a) {
  release_successor();
  after_predecessor();
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int hq = (int)(item % a.Hq);
  const long long t = item / a.Hq;
  const int s = (int)(t / a.max_q), i = (int)(t % a.max_q);
  if (s >= a.n_seqs) return;
  const int c0 = a.cu[s], c1 = a.cu[s + 1];
  if (!rows_in_range(a, c0, c1) || i >= c1 - c0) return;
  const float* part = static_cast<const float*>(a.c.ws) + (size_t)item * a.n_split * 132;
  const float mine = lane < a.n_split ? part[(size_t)lane * 132] : -INFINITY;
  const bool nan = __any_sync(0xffffffffu, isnan(mine));
  const float top = warp_max_xor(mine, 1);
  const float wt = mine == -INFINITY ? 0.f : expf(mine - top);
  const float sum = warp_sum_xor(wt, 1);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < a.n_split; ++k) {
    const float f = __shfl_sync(0xffffffffu, wt, k);
    if (__shfl_sync(0xffffffffu, mine, k) == -INFINITY) continue;   // saw no key
    const float4 p = *reinterpret_cast<const float4*>(part + (size_t)k * 132 + 4 + 4 * lane);
    acc.x = fmaf(f, p.x, acc.x);
    acc.y = fmaf(f, p.y, acc.y);
    acc.z = fmaf(f, p.z, acc.z);
    acc.w = fmaf(f, p.w, acc.w);
  }
  const float r = sum == 0.f ? 0.f : 1.f / sum;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * r, acc.y * r), hi = __floats2bfloat162_rn(acc.z * r, acc.w * r);
  const size_t row = ((size_t)c0 + i) * a.Hq + hq;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.c.out) + row * 128 + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (a.c.lse && lane == 0)
    a.c.lse[row] = nan ? __uint_as_float(0x7FC00000u) : (sum == 0.f ? -INFINITY : top + logf(sum));
}

// of a sequence, at most; one where the bound is 0, which looks at the sequence's count
long long q_blocks(const Pool& p, int max_q) { return std::max(((long long)max_q * p.G + 2 * kRows - 1) / (2 * kRows), 1ll); }

// Splits of the keys: where the blocks of rows fill less than half of the SMs,
// as many as fit in one wave, of at least four tiles each.
int splits(const Pool& p, int n_seqs, int max_q, long long max_len, int window, int n_sink) {
  long long keys = max_len;
  if (window) keys = std::min(keys, (long long)window + n_sink + std::min<long long>(max_q, 2 * kRows / p.G) + 2 * kKeys);
  const long long tiles = (keys + kKeys - 1) / kKeys, blocks = q_blocks(p, max_q) * n_seqs * p.cfg.num_kv_heads;
  if (max_q == 0) return 1;
  return (int)std::max(1ll, std::min<long long>({p.sm_count / blocks, tiles / 4, kMaxSplits}));
}

}  // namespace

size_t prefill_fp8_workspace(const Pool& p, int n_seqs, int max_q, int max_len) {
  const int n = splits(p, n_seqs, max_q, max_len, 0, 0);
  return n == 1 ? 16 : (size_t)n_seqs * max_q * p.cfg.num_q_heads * n * 132 * sizeof(float);
}

// Fewer blocks of rows are split further: the most that any call up to these bounds
// needs.  Only calls of up to half as many blocks as SMs are split; among those of as
// many blocks of queries the one with the most queries needs the most.
size_t prefill_fp8_workspace_up_to(const Pool& p, int n_seqs, int max_q, int max_len) {
  size_t most = 16;
  const int few = p.sm_count / 2;
  for (int b = 1; b <= std::min<long long>(few, q_blocks(p, max_q)); ++b)
    for (int s = 1; s <= std::min(few / b, n_seqs); ++s)
      most = std::max(most, prefill_fp8_workspace(p, s, std::min(max_q, b * 2 * kRows / p.G), max_len));
  return most;
}

cudaError_t launch_prefill_fp8(const Pool& p, const Fp8Store& f, int layer, int n_seqs, const int32_t* cu_q,
                               int max_q, const AttnCall& c, cudaStream_t s) {
  PrefillFp8Args a{fp8_layer(p, f, layer), c, cu_q, n_seqs, max_q, p.cfg.num_q_heads, p.G,
                   splits(p, n_seqs, max_q, c.max_len, c.window, c.n_sink), (int)q_blocks(p, max_q), p.err,
                   p.test_wait_polls > 0 ? p.test_wait_polls : kPolls, p.test_stall_first_copy};
  const long long ctas = (long long)a.q_blocks * n_seqs * a.L.Hkv * a.n_split;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(prefill_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(prefill_fp8_kernel, dim3((unsigned)ctas), kThreads, kSmem, s, 1, a);
  if (e != cudaSuccess || a.n_split == 1) return e;
  return launch_dependent(prefill_join_kernel, dim3((unsigned)(((long long)n_seqs * max_q * a.Hq + 7) / 8)), 256, 0, s, 1, a);
}

}  // namespace kvint2
