// The attention of one query row over the 8-bit cache, key by key: the plain
// form of what the tensor-core kernels compute.
#pragma once

#include <cuda_fp8.h>

#include "kv_device.cuh"
#include "kv_fp8.h"

namespace kvint2 {

__device__ __forceinline__ float4 e4m3x4_f32(uint32_t w) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
  return make_float4(x.x, x.y, y.x, y.y);
}

// One warp: lane owns channels 4 lane .. 4 lane + 3 of the row.
__device__ __forceinline__ void attend_row(const Fp8Layer& L, const int32_t* pt, int max_pages, int h,
                                           const uint16_t* q, int pos, int window, int n_sink, float scale,
                                           uint16_t* out, float* lse, int* err, int lane) {
  const int c = 4 * lane, per = L.P / kTile;
  const uint2 qw = *reinterpret_cast<const uint2*>(q + c);
  const float q0 = bf16lo(qw.x), q1 = bf16hi(qw.x), q2 = bf16lo(qw.y), q3 = bf16hi(qw.y);
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
  const int low = window ? max(pos - window + 1, 0) : 0;
  for (int j0 = 0; j0 <= pos; j0 += kTile) {
    if (j0 + kTile <= low && j0 >= n_sink) {
      j0 = low / kTile * kTile - kTile;
      continue;
    }
    const int pid = pt[j0 / L.P];
    if (pid < 0 || pid >= L.num_pages) {
      flag_error(err, KV_DEVERR_PAGE_ID);
      continue;
    }
    const size_t tile = ((size_t)pid * L.Hkv + h) * per + j0 / kTile % per;
    const uint8_t* codes = L.codes + tile * kFp8TileBytes;
    const float ks = ldexpf(scale, L.exps[tile * 2]), vs = ldexpf(1.f, L.exps[tile * 2 + 1]);
    for (int t = 0; t < kTile; ++t) {
      const int j = j0 + t;
      if (j > pos || (j < low && j >= n_sink)) continue;
      const float4 k = e4m3x4_f32(
          *reinterpret_cast<const uint32_t*>(codes + (t >> 3) * 1024 + (c >> 6) * 512 + (t & 7) * 64 + (c & 63)));
      const float x = ks * warp_sum_xor(q0 * k.x + q1 * k.y + q2 * k.z + q3 * k.w, 1);
      const float4 v = e4m3x4_f32(*reinterpret_cast<const uint32_t*>(
          codes + 2048 + ((t & 1) + 2 * (t >> 3)) * 512 + (c >> 4) * 64 + ((t & 7) >> 1) * 16 + (c & 15)));
      const float mn = fmaxf(m, x), f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(x - mn), w = p * vs;
      l = l * f + p;
      o0 = o0 * f + w * v.x;
      o1 = o1 * f + w * v.y;
      o2 = o2 * f + w * v.z;
      o3 = o3 * f + w * v.w;
      m = mn;
    }
  }
  const float r = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
  const __nv_bfloat162 a = __floats2bfloat162_rn(o0 * r, o1 * r), b = __floats2bfloat162_rn(o2 * r, o3 * r);
  *reinterpret_cast<uint2*>(out + c) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (lse && lane == 0) *lse = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace kvint2
