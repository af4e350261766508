// Gradient norm and AdamW over many tensors in one launch.
//
// The tensors' pointers and sizes travel as kernel parameters (at most kAdamCap or kNormCap per
// launch), so nothing is copied to the device first and the caller's arrays are free when the
// call returns.  Every tensor is cut into chunks; a block finds its chunk's tensor by binary
// search over the running chunk counts.
#include <algorithm>
#include <cmath>

#include <cuda_fp16.h>

#include "mok_mx.cuh"
#include "mok_vec.cuh"

namespace mok {

// ------------------------------------------------------------------ gradient norm
constexpr int kOptThreads = 256;
constexpr int kNormChunk = 16384;   // elements per chunk of the gradient norm
constexpr int kNormCap = 1024;      // tensors per launch
constexpr int kNormCapSmall = 64;
constexpr int kNormBlocksPerSm = 8;

template <int CAP>
struct NormTable {
  const void* grad[CAP];
  int64_t numel[CAP];
  uint32_t end[CAP];  // chunks up to and including this tensor
  uint8_t f32[CAP];
  int n;
  uint32_t chunks;
  float* partial;     // one per block
};

template <class Table>
__device__ __forceinline__ int tensor_of(const Table& p, uint32_t chunk) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.end[mid] <= chunk) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

template <bool F32>
__device__ __forceinline__ float square_sum(const void* g, int64_t numel, int64_t at) {
  float a = 0.0f;
  const int64_t end = min(numel, at + kNormChunk);
  for (int64_t i = at + 8 * threadIdx.x; i < end; i += 8 * kOptThreads) {
    if (i + 8 <= numel) {
      const Vec8 v = load8<F32>(g, i >> 3);
#pragma unroll
      for (int j = 0; j < 8; ++j) a = fmaf(v.v[j], v.v[j], a);
    } else {
      for (int64_t q = i; q < numel; ++q) {
        const float v = F32 ? static_cast<const float*>(g)[q] : __bfloat162float(static_cast<const __nv_bfloat16*>(g)[q]);
        a = fmaf(v, v, a);
      }
    }
  }
  return a;
}

template <int CAP>
__global__ void __launch_bounds__(kOptThreads) grad_norm_kernel(const __grid_constant__ NormTable<CAP> p) {
  __shared__ float smem[kOptThreads / 32];
  float a = 0.0f;
  for (uint32_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const int t = tensor_of(p, c);
    const int64_t at = (int64_t)(c - (t ? p.end[t - 1] : 0u)) * kNormChunk;
    a += p.f32[t] ? square_sum<true>(p.grad[t], p.numel[t], at) : square_sum<false>(p.grad[t], p.numel[t], at);
  }
  a = warp_sum(a);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < kOptThreads / 32; ++w) s += smem[w];
    p.partial[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(256) grad_norm_join_kernel(const float* __restrict__ partial, int n,
                                                             float max_norm, float* __restrict__ out) {
  __shared__ double smem[8];
  double a = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) a += partial[i];
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) a += smem[w];
    const float norm = (float)sqrt(a);
    out[0] = norm;
    out[1] = !isfinite(norm) ? NAN : max_norm > 0.0f ? fminf(1.0f, max_norm / norm) : 1.0f;
  }
}

// ------------------------------------------------------------------ AdamW
constexpr int kAdamChunk = 4096;  // elements per block
constexpr int kAdamCap = 384;     // tensors per launch: about 30 KB of the 32 KB of parameters
constexpr int kAdamCapSmall = 24;

struct AdamEntry {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t numel;
  float decay;
  int32_t param_f32, grad_f32;
};

struct AdamHyper {
  float lr, b1, b2, omb1, omb2, c1, c2, eps;  // omb = 1 - b, c = 1 / (1 - b^step)
  uint32_t turn;                              // 0x9E3779B9 step
};

template <int CAP>
struct AdamTable {
  AdamEntry t[CAP];
  uint32_t end[CAP];
  int n;
  AdamHyper h;
  const float* clip;
};

// Eight consecutive elements from `i` of which `n` exist (the others read as 0, are not written).
template <bool F32>
__device__ __forceinline__ Vec8 load8n(const void* p, int64_t i, int n) {
  if (n >= 8) return load8<F32>(p, i >> 3);
  Vec8 a;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    a.v[j] = j >= n ? 0.0f : F32 ? static_cast<const float*>(p)[i + j] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i + j]);
  return a;
}
template <bool F32>
__device__ __forceinline__ void store8n(void* p, int64_t i, int n, const Vec8& a) {
  if (n >= 8) {
    store8<F32>(p, i >> 3, a);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if (F32) static_cast<float*>(p)[i + j] = a.v[j];
      else static_cast<__nv_bfloat16*>(p)[i + j] = __float2bfloat16_rn(a.v[j]);
    }
}

// Four E4M3 codes to fp32 (exact, by way of f16).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float* o) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)c));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(c >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
}
// 2^(b - 127) of a scale byte (b = 0: 2^-127, a subnormal).
__device__ __forceinline__ float e8m0(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x400000u); }

__device__ __forceinline__ Vec8 load_state8(const void* codes, const uint8_t* scales, int64_t i, int n) {
  uint2 c = make_uint2(0, 0);
  if (n >= 8) {
    c = static_cast<const uint2*>(codes)[i >> 3];
  } else {
    for (int j = 0; j < n; ++j) {
      const uint32_t b = static_cast<const uint8_t*>(codes)[i + j];
      if (j < 4) c.x |= b << (8 * j);
      else c.y |= b << (8 * (j - 4));
    }
  }
  const float s = n > 0 ? e8m0(scales[i >> 5]) : 0.0f;
  Vec8 a;
  e4m3x4_to_f32(c.x, a.v);
  e4m3x4_to_f32(c.y, a.v + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) a.v[j] *= s;
  return a;
}

// 32 bits for element i at this step: a multiply-and-shift mixer, so that neither neighbouring
// elements nor consecutive steps are correlated (a plain multiple of the step is: averages then
// drift by some percent).
__device__ __forceinline__ uint32_t dither_bits(uint32_t i, uint32_t turn) {
  uint32_t x = 0x85EBCA6Bu * i + turn;
  x = (x ^ (x >> 15)) * 0x2C1B3C6Du;
  x = (x ^ (x >> 12)) * 0x297A2D39u;
  return x ^ (x >> 15);
}
// Dithered rounding of 0 <= q <= 448 to E4M3: up when the place between the two codes plus
// (r + 1/2) / 2^16 reaches 1.  Normal codes keep 3 bits of mantissa, codes below 2^-6 are
// multiples of 2^-9.
__device__ __forceinline__ float dither_e4m3(float q, uint32_t r) {
  const float normal = __uint_as_float((__float_as_uint(q) + (r << 4) + 8u) & 0xFFF00000u);
  const float small = floorf(q * 512.0f + ((float)r + 0.5f) * 0x1p-16f) * 0x1p-9f;
  return q < 0x1p-6f ? small : fminf(normal, 448.0f);
}

// All 32 lanes call this: four lanes share a block of 32 elements.
// V: the second moment.
template <bool V>
__device__ __forceinline__ void store_state8(void* codes, uint8_t* scales, int64_t i, int n, const Vec8& a, uint32_t turn) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(a.v[j]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int s = mx_exponent(amax);
  const float inv = __uint_as_float((uint32_t)(127 - s) << 23);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t r = dither_bits((uint32_t)i + j, turn);
    q[j] = dither_e4m3(fabsf(a.v[j]) * inv, V ? r & 0xFFFFu : r >> 16);
    if (V && a.v[j] > 0.0f) q[j] = fmaxf(q[j], 0x1p-9f);
    q[j] = copysignf(q[j], a.v[j]);
  }
  const uint32_t lo = e4m3x2(q[0], q[1]) | (uint32_t)e4m3x2(q[2], q[3]) << 16;
  const uint32_t hi = e4m3x2(q[4], q[5]) | (uint32_t)e4m3x2(q[6], q[7]) << 16;
  if (n >= 8) {
    static_cast<uint2*>(codes)[i >> 3] = make_uint2(lo, hi);
  } else {
    for (int j = 0; j < n; ++j) static_cast<uint8_t*>(codes)[i + j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
  }
  if (n > 0 && (i & 31) == 0) scales[i >> 5] = (uint8_t)(s + 127);
}

template <bool MX, bool P32, bool G32>
__device__ __forceinline__ void adam_chunk(const AdamEntry& t, const AdamHyper& h, float clip, int64_t at) {
#pragma unroll 1
  for (int u = 0; u < kAdamChunk; u += 8 * kOptThreads) {
    const int64_t i = at + u + 8 * threadIdx.x;
    const int n = (int)min((int64_t)8, t.numel - i);  // may be <= 0: such lanes only take part in the shuffles
    if (!MX && n <= 0) return;
    Vec8 g = load8n<G32>(t.grad, i, n);
    Vec8 w = load8n<true>(P32 ? t.param : t.master, i, n);
    Vec8 m, v;
    if constexpr (MX) {
      m = load_state8(t.m, t.ms, i, n);
      v = load_state8(t.v, t.vs, i, n);
    } else {
      m = load8n<true>(t.m, i, n);
      v = load8n<true>(t.v, i, n);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = g.v[j] * clip;
      m.v[j] = h.b1 * m.v[j] + h.omb1 * gj;
      v.v[j] = h.b2 * v.v[j] + h.omb2 * (gj * gj);
      const float step = (m.v[j] * h.c1) / (sqrtf(v.v[j] * h.c2) + h.eps);
      w.v[j] -= h.lr * (step + t.decay * w.v[j]);
    }
    if constexpr (MX) {
      store_state8<false>(t.m, t.ms, i, n, m, h.turn);
      store_state8<true>(t.v, t.vs, i, n, v, h.turn);
    } else {
      store8n<true>(t.m, i, n, m);
      store8n<true>(t.v, i, n, v);
    }
    store8n<true>(P32 ? t.param : t.master, i, n, w);
    if constexpr (!P32) store8n<false>(t.param, i, n, w);
  }
}

template <int CAP, bool MX>
__global__ void __launch_bounds__(kOptThreads) adamw_kernel(const __grid_constant__ AdamTable<CAP> p) {
  const float clip = p.clip ? p.clip[1] : 1.0f;
  if (clip != clip) return;  // the gradients' norm is not finite: nothing changes
  const int k = tensor_of(p, blockIdx.x);
  const AdamEntry& t = p.t[k];
  const int64_t at = (int64_t)(blockIdx.x - (k ? p.end[k - 1] : 0u)) * kAdamChunk;
  if (t.param_f32) {
    if (t.grad_f32) adam_chunk<MX, true, true>(t, p.h, clip, at);
    else adam_chunk<MX, true, false>(t, p.h, clip, at);
  } else {
    if (t.grad_f32) adam_chunk<MX, false, true>(t, p.h, clip, at);
    else adam_chunk<MX, false, false>(t, p.h, clip, at);
  }
}

// ------------------------------------------------------------------ host
static int64_t chunks_of(int64_t numel, int chunk) { return (numel + chunk - 1) / chunk; }
static bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int64_t kMaxNumel = int64_t(1) << 40;  // 2^40 elements: chunk counts stay below 2^31

// Launches of the gradient norm: tensors are taken in order, kNormCap per launch.
static bool norm_counts(int n, const int64_t* numel, int64_t* blocks) {
  *blocks = 0;
  const int64_t most = (int64_t)num_sms() * kNormBlocksPerSm;
  for (int i = 0; i < n; i += kNormCap) {
    int64_t c = 0;
    for (int j = i; j < std::min(n, i + kNormCap); ++j) {
      if (numel[j] < 0 || numel[j] > kMaxNumel) return false;
      c += chunks_of(numel[j], kNormChunk);
    }
    if (c > 0x7fffffffLL) return false;
    *blocks += std::min(c, most);
  }
  return *blocks < 0x7fffffffLL;
}

template <int CAP>
static cudaError_t launch_norm(int n, const void* const* grads, const int64_t* numel, const int32_t* types,
                               float* partial, int* blocks, cudaStream_t s) {
  NormTable<CAP> p;
  int64_t c = 0;
  p.n = n;
  for (int j = 0; j < n; ++j) {
    c += chunks_of(numel[j], kNormChunk);
    p.grad[j] = grads[j];
    p.numel[j] = numel[j];
    p.end[j] = (uint32_t)c;
    p.f32[j] = types[j] == MOK_T_F32;
  }
  p.chunks = (uint32_t)c;
  p.partial = partial;
  *blocks = (int)std::min<int64_t>(c, (int64_t)num_sms() * kNormBlocksPerSm);
  if (*blocks == 0) return cudaSuccess;
  prof_begin("grad_norm", s);
  grad_norm_kernel<CAP><<<*blocks, kOptThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

template <int CAP, bool MX>
static cudaError_t launch_adam(int n, const mok_adamw_tensor* t, const AdamHyper& h, const float* clip, cudaStream_t s, int* launches) {
  AdamTable<CAP> p;
  int64_t c = 0;
  p.n = n;
  p.h = h;
  p.clip = clip;
  for (int j = 0; j < n; ++j) {
    c += chunks_of(t[j].numel, kAdamChunk);
    p.t[j] = AdamEntry{t[j].param, t[j].grad, t[j].master, t[j].exp_avg, t[j].exp_avg_sq, t[j].exp_avg_scale,
                       t[j].exp_avg_sq_scale, t[j].numel, (float)t[j].weight_decay, t[j].param_type == MOK_T_F32,
                       t[j].grad_type == MOK_T_F32};
    p.end[j] = (uint32_t)c;
  }
  if (c == 0) return cudaSuccess;
  prof_begin("adamw", s);
  adamw_kernel<CAP, MX><<<(unsigned)c, kOptThreads, 0, s>>>(p);
  prof_end(s);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace mok

extern "C" {

size_t mok_grad_norm_workspace_size(int n_tensors, const int64_t* numel) {
  using namespace mok;
  int64_t blocks;
  if (n_tensors < 0 || (n_tensors > 0 && !numel) || !norm_counts(n_tensors, numel, &blocks)) return 0;
  return 256 + sizeof(float) * (size_t)std::max<int64_t>(blocks, 1);
}

int mok_grad_norm(int n_tensors, const void* const* grads, const int64_t* numel,
                  const int32_t* types, float max_norm, float* out, void* ws, size_t ws_bytes,
                  mok_stream_t stream) {
  using namespace mok;
  if (n_tensors < 0 || (n_tensors > 0 && (!grads || !numel || !types)) || !out || !ws || max_norm != max_norm)
    return MOK_ERR_INVALID_ARG;
  for (int i = 0; i < n_tensors; ++i) {
    if (numel[i] < 0 || (numel[i] > 0 && !grads[i]) || (types[i] != MOK_T_BF16 && types[i] != MOK_T_F32))
      return MOK_ERR_INVALID_ARG;
    if (!is16(grads[i])) return MOK_ERR_UNSUPPORTED;
  }
  if (!is16(ws)) return MOK_ERR_UNSUPPORTED;
  const size_t need = mok_grad_norm_workspace_size(n_tensors, numel);
  if (need == 0) return MOK_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  int total = 0, launches = 0;
  for (int i = 0; i < n_tensors; i += kNormCap) {
    const int n = std::min(n_tensors - i, kNormCap);
    int blocks = 0;
    const cudaError_t e = n <= kNormCapSmall
        ? launch_norm<kNormCapSmall>(n, grads + i, numel + i, types + i, partial + total, &blocks, s)
        : launch_norm<kNormCap>(n, grads + i, numel + i, types + i, partial + total, &blocks, s);
    if (e != cudaSuccess) return MOK_ERR_CUDA;
    total += blocks;
    launches += blocks > 0;
  }
  prof_begin("grad_norm_join", s);
  grad_norm_join_kernel<<<1, 256, 0, s>>>(partial, total, max_norm, out);
  prof_end(s);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(launches + 1);
  return MOK_OK;
}

int mok_adamw_step(const mok_adamw_args* args, const mok_adamw_tensor* tensors, int n_tensors,
                   const float* clip, mok_stream_t stream) {
  using namespace mok;
  if (!args || n_tensors < 0 || (n_tensors > 0 && !tensors)) return MOK_ERR_INVALID_ARG;
  const mok_adamw_args& a = *args;
  if (!(a.beta1 >= 0.0 && a.beta1 < 1.0) || !(a.beta2 >= 0.0 && a.beta2 < 1.0) || !(a.eps > 0.0) ||
      !std::isfinite(a.eps) || !std::isfinite(a.lr) || a.step < 1 ||
      (a.state_format != MOK_STATE_F32 && a.state_format != MOK_STATE_MXFP8))
    return MOK_ERR_INVALID_ARG;
  const bool mx = a.state_format == MOK_STATE_MXFP8;
  for (int i = 0; i < n_tensors; ++i) {
    const mok_adamw_tensor& t = tensors[i];
    if (t.numel < 0 || (t.param_type != MOK_T_BF16 && t.param_type != MOK_T_F32) ||
        (t.grad_type != MOK_T_BF16 && t.grad_type != MOK_T_F32) || !std::isfinite(t.weight_decay))
      return MOK_ERR_INVALID_ARG;
    if (t.numel > kMaxNumel) return MOK_ERR_UNSUPPORTED;
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || (t.param_type == MOK_T_BF16) != (t.master != nullptr) ||
        (mx && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
      return MOK_ERR_INVALID_ARG;
    for (const void* q : {(const void*)t.param, t.grad, (const void*)t.master, (const void*)t.exp_avg, (const void*)t.exp_avg_sq})
      if (!is16(q)) return MOK_ERR_UNSUPPORTED;
  }
  set_last_launches(0);
  AdamHyper h;
  h.lr = (float)a.lr;
  h.b1 = (float)a.beta1;
  h.b2 = (float)a.beta2;
  h.omb1 = (float)(1.0 - a.beta1);
  h.omb2 = (float)(1.0 - a.beta2);
  h.c1 = (float)(1.0 / (1.0 - std::pow(a.beta1, (double)a.step)));
  h.c2 = (float)(1.0 / (1.0 - std::pow(a.beta2, (double)a.step)));
  h.eps = (float)a.eps;
  h.turn = 0x9E3779B9u * (uint32_t)a.step;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int launches = 0;
  for (int i = 0; i < n_tensors; i += kAdamCap) {
    const int n = std::min(n_tensors - i, kAdamCap);
    const bool small = n <= kAdamCapSmall;
    const cudaError_t e =
        mx ? (small ? launch_adam<kAdamCapSmall, true>(n, tensors + i, h, clip, s, &launches)
                    : launch_adam<kAdamCap, true>(n, tensors + i, h, clip, s, &launches))
           : (small ? launch_adam<kAdamCapSmall, false>(n, tensors + i, h, clip, s, &launches)
                    : launch_adam<kAdamCap, false>(n, tensors + i, h, clip, s, &launches));
    if (e != cudaSuccess) return MOK_ERR_CUDA;
  }
  set_last_launches(launches);
  return MOK_OK;
}

}  // extern "C"
