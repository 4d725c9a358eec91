// What the prompt attention kernels share: tcgen05 and barrier wrappers, paired fp32
// arithmetic, bounded waits that end every role together.
#pragma once

#include "kv_device.cuh"

namespace kvint2 {

constexpr uint32_t kOperand = 128 * 256;       // a 128 x 128 operand of two bytes a value

// Shared-memory operand of 128-byte rows in the 128-byte swizzle (8-row atoms of
// 1024 bytes).  K-major (Q, K): the leading offset is unused.  MN-major (V: rows
// are tokens, 64 channels each): leading offset = the second 64 channels,
// stride offset = the next 8 tokens.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lead) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define KV_TIE8(v, i) \
  "+f"((v)[i]), "+f"((v)[i + 1]), "+f"((v)[i + 2]), "+f"((v)[i + 3]), "+f"((v)[i + 4]), "+f"((v)[i + 5]), \
      "+f"((v)[i + 6]), "+f"((v)[i + 7])
// 32 columns of this thread's row; the values are there after settle()
__device__ __forceinline__ void ld32(uint32_t t, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(t)
      : "memory");
}
// 16 columns
__device__ __forceinline__ void ld16(uint32_t t, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void settle16(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KV_TIE8(v, 0), KV_TIE8(v, 8) : : "memory");
}
// no use of the values moves above the wait
__device__ __forceinline__ void settle(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : KV_TIE8(v, 0), KV_TIE8(v, 8), KV_TIE8(v, 16), KV_TIE8(v, 24)
               :
               : "memory");
}
__device__ __forceinline__ void st16(uint32_t t, const uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
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
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits [0, x) of a word that starts at bit `from`.
__device__ __forceinline__ uint32_t below(int x, int from) {
  const int n = x - from;
  return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}

// Waits of the roles of a CTA.
struct Waiter {
  int* abort;
  int polls;
  const int* steps;                            // of the walker
  // whether the phase with `parity` completed; a wait that runs out ends every role
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    for (int i = 0; !mbar_wait(bar, parity, 1); ++i) {
      if ((i & 63) == 63 && (i >= polls || *reinterpret_cast<volatile int*>(abort))) {
        *reinterpret_cast<volatile int*>(abort) = 1;
        return false;
      }
    }
    return true;
  }
  // The same for what the walker hands over: the limit starts again while it passes blocks
  // without rows (3 ns each over the device: 6 s for the largest grid).
  __device__ __forceinline__ bool handed(uint64_t* bar, uint32_t parity) const {
    int seen = -1;
    for (int i = 0; !mbar_wait(bar, parity, 1); ++i) {
      if ((i & 63) != 63) continue;
      const int now = *reinterpret_cast<const volatile int*>(steps);
      if (*reinterpret_cast<volatile int*>(abort) || (i >= polls && now == seen)) {
        *reinterpret_cast<volatile int*>(abort) = 1;
        return false;
      }
      if (now != seen) i = 0;
      seen = now;
    }
    return true;
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.b32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}

}  // namespace kvint2
