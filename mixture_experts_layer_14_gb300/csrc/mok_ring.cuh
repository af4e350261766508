// Rows of bf16 or fp32 elements, eight at a time: raw vectors, a ring of rows in shared memory that a
// thread fills by asynchronous copies of exactly what it reads back itself, and pairs for the
// two-wide fp32 instructions.
#pragma once

#include <cuda_fp16.h>

#include "mok_mx.cuh"
#include "mok_vec.cuh"

namespace mok {

// Eight elements as they are stored: bf16 in one register quadruple, fp32 in two.
template <bool F32>
struct Raw8 {
  uint4 u[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> raw8(const void* p, int64_t i) {
  Raw8<F32> r;
  if constexpr (F32) {
    r.u[0] = static_cast<const uint4*>(p)[2 * i];
    r.u[1] = static_cast<const uint4*>(p)[2 * i + 1];
  } else {
    r.u[0] = static_cast<const uint4*>(p)[i];
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> zero8() {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.u[i] = make_uint4(0, 0, 0, 0);
  return r;
}
template <bool F32>
__device__ __forceinline__ Vec8 value8(const Raw8<F32>& r) {
  if constexpr (F32)
    return {__uint_as_float(r.u[0].x), __uint_as_float(r.u[0].y), __uint_as_float(r.u[0].z), __uint_as_float(r.u[0].w),
            __uint_as_float(r.u[1].x), __uint_as_float(r.u[1].y), __uint_as_float(r.u[1].z), __uint_as_float(r.u[1].w)};
  else
    return unpack8(r.u[0]);
}

// Vector v of a row that begins at vector `row` of the array, to the ring's place `at` (bytes): bf16
// in one plane of 16 bytes per vector; fp32 in two, through L1, because each copy uses half a
// sector (past L1, or with the halves of a warp's vectors redistributed, 10-25% slower).
template <bool F32>
__device__ __forceinline__ void copy8(uint32_t at, const void* p, int64_t row, int v, int nvec) {
  if (v >= nvec) return;
  if constexpr (F32) {
    copy16_ca(at + 16 * v, static_cast<const uint4*>(p) + 2 * (row + v));
    copy16_ca(at + 16 * (nvec + v), static_cast<const uint4*>(p) + 2 * (row + v) + 1);
  } else {
    copy16(at + 16 * v, static_cast<const uint4*>(p) + row + v);
  }
}
__device__ __forceinline__ uint4 ring16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at));
  return u;
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> ring8(uint32_t at, int v, int nvec) {
  Raw8<F32> r;
  r.u[0] = ring16(at + 16 * v);
  if constexpr (F32) r.u[1] = ring16(at + 16 * (nvec + v));
  return r;
}
__device__ __forceinline__ Vec8 load_weight(const void* w, int f32, int v, bool in) {
  if (!in) return {};
  return f32 ? load8<true>(w, v) : load8<false>(w, v);
}

// 2^(byte - 127): a UE8M0 scale (255, which no block has, gives infinity).
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }
__device__ __forceinline__ uint4 e4m3_halves(uint2 q) {  // as f16, which holds every E4M3 value
  uint4 r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.x) : "h"((uint16_t)q.x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.y) : "h"((uint16_t)(q.x >> 16)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.z) : "h"((uint16_t)q.y));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.w) : "h"((uint16_t)(q.y >> 16)));
  return r;
}
// Values of eight E4M3 codes times their block's scale (every product is exact but where it leaves
// fp32's range).
__device__ __forceinline__ Vec8 dequantise8(uint2 q, float scale) {
  Vec8 r;
  const uint4 u = e4m3_halves(q);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    r.v[2 * i] = f.x * scale;
    r.v[2 * i + 1] = f.y * scale;
  }
  return r;
}

// Eight values as four pairs, for the two-wide fp32 instructions: with scalar ones the RMS
// norm's backward pass takes 360 instructions per warp and row, three quarters of the issue slots.
struct Pairs {
  float2 p[4];
};
__device__ __forceinline__ Pairs pairs(const Vec8& a) {
  Pairs r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.p[j] = make_float2(a.v[2 * j], a.v[2 * j + 1]);
  return r;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
template <bool F32>
__device__ __forceinline__ void store_pairs(void* p, int64_t i, const Pairs& a) {
  store8<F32>(p, i, {a.p[0].x, a.p[0].y, a.p[1].x, a.p[1].y, a.p[2].x, a.p[2].y, a.p[3].x, a.p[3].y});
}

// The scale byte s + 127 of a block with this largest magnitude, s the smallest integer with amax <= 448
// 2^s = 1.75 2^(s + 8): the exponent less 8, and one more for mantissas above 1.75, which the sum
// carries over.  (mx_exponent without its cases: subnormal numbers give 0 all the same.)
__device__ __forceinline__ int mx_scale_byte(float amax) {
  return max((int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8, 0);
}
__device__ __forceinline__ uint2 mx_codes8(const Pairs& a, int byte) {
  const float2 inv = both(__uint_as_float((uint32_t)(254 - byte) << 23));  // 2^-s
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = __fmul2_rn(a.p[j], inv);
    q[j] = e4m3x2(v.x, v.y);
  }
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

}  // namespace mok
