// Eight consecutive elements of a row, as the bandwidth-bound kernels around the layer hold them:
// loads from and stores to bf16 (16 bytes) and fp32 (32 bytes), and sums over a warp.
#pragma once

#include "mok_device.cuh"

namespace mok {

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ Vec8 unpack8(uint4 u) {
  return {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
          bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
}
__device__ __forceinline__ uint4 pack8(const Vec8& a) {
  return make_uint4(pack_bf16x2(a.v[0], a.v[1]), pack_bf16x2(a.v[2], a.v[3]),
                    pack_bf16x2(a.v[4], a.v[5]), pack_bf16x2(a.v[6], a.v[7]));
}
// Vector `i` (elements 8 i ..) of a bf16 or fp32 array.
template <bool F32>
__device__ __forceinline__ Vec8 load8(const void* p, int64_t i) {
  if constexpr (F32) {
    const float4 a = static_cast<const float4*>(p)[2 * i], b = static_cast<const float4*>(p)[2 * i + 1];
    return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  } else {
    return unpack8(static_cast<const uint4*>(p)[i]);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const Vec8& a) {
  if constexpr (F32) {
    static_cast<float4*>(p)[2 * i] = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
    static_cast<float4*>(p)[2 * i + 1] = make_float4(a.v[4], a.v[5], a.v[6], a.v[7]);
  } else {
    static_cast<uint4*>(p)[i] = pack8(a);
  }
}

// Asynchronous 16-byte copies to shared memory, in groups; copies_wait<N> waits until all but this
// thread's newest N groups have landed (it sees only its own: a thread that reads back exactly
// what it copied needs no barrier).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_ca(uint32_t dst, const void* src) {  // through L1
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Launches a kernel that may begin while the one before it in the stream still runs; it waits
// with griddepcontrol.wait before it touches that one's results.
template <class... P, class... A>
cudaError_t launch_after_smem(int smem, void (*kernel)(P...), int grid, int block, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)block);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int block, cudaStream_t s, A... args) {
  return launch_after_smem(0, kernel, grid, block, s, args...);
}

}  // namespace mok
