// Device helpers of the 4-bit key/value cache (layout and value definition in
// include/gdn.h): record offsets, page lookup, e2m1 / e4m3 conversions.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "gdn_common.cuh"

namespace gdn {
namespace kv4 {

constexpr int kRec = 32;  // tokens in a record

// Byte offsets inside a record of head size D.
__host__ __device__ constexpr int rec_bytes(int D) { return 36 * D; }
__host__ __device__ constexpr int off_v(int D) { return 16 * D; }
__host__ __device__ constexpr int off_ks(int D) { return 32 * D; }
__host__ __device__ constexpr int off_vs(int D) { return 34 * D; }

// A length as it counts: one out of range as 0 (and is reported by whoever passes `report_it`).
__device__ __forceinline__ int check_len(const gdn_kv4_cache& c, int n, bool report_it) {
  if (n < 0 || (int64_t)n > (int64_t)c.max_pages * c.page_tokens) {
    if (report_it) report(c.status, GDN_ERR_ROW_RANGE);
    return 0;
  }
  return n;
}

// Length of sequence b.
__device__ __forceinline__ int seq_len(const gdn_kv4_cache& c, int b, bool report_it) {
  return check_len(c, c.kv_len[b], report_it);
}

// The record of head h that holds position `pos` of sequence b, or NULL when
// the page number is outside the pool.
__device__ __forceinline__ uint8_t* record(const gdn_kv4_cache& c, int b, int h, int pos) {
  const int page = c.table[(int64_t)b * c.table_stride + pos / c.page_tokens];
  if (page < 0 || page >= c.n_pages) return nullptr;
  const int recs = c.page_tokens / kRec;
  return static_cast<uint8_t*>(c.pages) + (int64_t)page * c.page_stride +
         ((int64_t)h * recs + (pos % c.page_tokens) / kRec) * rec_bytes(c.D);
}

// Byte `i` (0..3) of w as two e2m1 codes -> two binary16 values, low half first.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2(uint32_t w) {
  uint32_t d;
  if constexpr (I == 0)
    asm("{.reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(d) : "r"(w));
  if constexpr (I == 1)
    asm("{.reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w));
  if constexpr (I == 2)
    asm("{.reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(d) : "r"(w));
  if constexpr (I == 3)
    asm("{.reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, e;}" : "=r"(d) : "r"(w));
  return d;
}

// Two e4m3 bytes (low 16 bits of w) -> two binary16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {
  uint32_t d;
  asm("{.reg .b16 a,b; mov.b32 {a,b}, %1; cvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(d) : "r"(w));
  return d;
}

__device__ __forceinline__ float e4m3(uint8_t s) {
  const uint32_t h = e4m3x2(s);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// fp32 -> e4m3, nearest even, saturating.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(x));
  return d & 0xffu;
}

// Two fp32 values -> a byte of two e2m1 codes (first one in the low half),
// nearest even, saturating.
__device__ __forceinline__ uint32_t to_e2m1x2(float first, float second) {
  uint32_t d;
  asm("{.reg .b8 a; cvt.rn.satfinite.e2m1x2.f32 a, %1, %2; mov.b32 %0, {a, 0, 0, 0};}"
      : "=r"(d)
      : "f"(second), "f"(first));
  return d;
}

// value of e2m1 code `c` (0..15)
__device__ __forceinline__ float e2m1(uint32_t c) {
  const uint32_t h = e2m1x2<0>(c);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

template <int DT>
struct Elem;
template <>
struct Elem<GDN_F32> {
  using T = float;
  static __device__ __forceinline__ T from(float x) { return x; }
};
template <>
struct Elem<GDN_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ T from(float x) {
    uint16_t d;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(d) : "f"(x));
    return d;
  }
};
template <>
struct Elem<GDN_F16> {
  using T = uint16_t;
  static __device__ __forceinline__ T from(float x) { return __half_as_ushort(__float2half_rn(x)); }
};

template <int DT>
__device__ __forceinline__ float to_float(typename Elem<DT>::T x) {
  if constexpr (DT == GDN_F32) return x;
  if constexpr (DT == GDN_BF16) return __uint_as_float((uint32_t)x << 16);
  if constexpr (DT == GDN_F16) return __half2float(__ushort_as_half(x));
}

// 8 consecutive elements at p (16-byte aligned) as fp32.
template <int DT>
__device__ __forceinline__ void load8(const void* p, float (&x)[8]) {
  if constexpr (DT == GDN_F32) {
    const float4 a = ld_nc_f4(static_cast<const float*>(p));
    const float4 b = ld_nc_f4(static_cast<const float*>(p) + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 u = ld_nc_u4(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == GDN_BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
}

// Checks parent[0..N) (N <= 64) of one sequence; every thread may call it.
__device__ __forceinline__ bool tree_ok(const int32_t* parent, int N) {
  bool ok = parent[0] == -1;
#pragma unroll 4
  for (int n = 1; n < N; ++n) ok = ok && parent[n] >= 0 && parent[n] < n;
  return ok;
}

}  // namespace kv4
}  // namespace gdn
