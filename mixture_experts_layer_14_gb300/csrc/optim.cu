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

// Squares of the chunk at `at`, a thread's share.  Whole chunks go eight vectors at a time, all
// loaded before the first is used: one 16-byte load per thread in flight reads at 60% of the
// copy rate, eight at the full one.
template <bool F32>
__device__ __forceinline__ float square_sum(const void* g, int64_t numel, int64_t at) {
  constexpr int kBatch = F32 ? 4 : 8;
  float a[2] = {0.0f, 0.0f};
  if (at + kNormChunk <= numel) {
#pragma unroll 1
    for (int u = 0; u < kNormChunk / (8 * kOptThreads); u += kBatch) {
      const int64_t i = (at >> 3) + u * kOptThreads + threadIdx.x;
      uint4 raw[8];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if constexpr (F32) {
          raw[2 * b] = __ldcs(static_cast<const uint4*>(g) + 2 * (i + b * kOptThreads));
          raw[2 * b + 1] = __ldcs(static_cast<const uint4*>(g) + 2 * (i + b * kOptThreads) + 1);
        } else {
          raw[b] = __ldcs(static_cast<const uint4*>(g) + i + b * kOptThreads);
        }
      }
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if constexpr (F32) {
          const float v[4] = {__uint_as_float(raw[b].x), __uint_as_float(raw[b].y), __uint_as_float(raw[b].z), __uint_as_float(raw[b].w)};
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j & 1] = fmaf(v[j], v[j], a[j & 1]);
        } else {
          const Vec8 v = unpack8(raw[b]);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j & 1] = fmaf(v.v[j], v.v[j], a[j & 1]);
        }
      }
    }
  } else {
    for (int64_t i = at + 8 * threadIdx.x; i < numel; i += 8 * kOptThreads) {
      const Vec8 v = load8n<F32>(g, i, (int)min((int64_t)8, numel - i));
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j & 1] = fmaf(v.v[j], v.v[j], a[j & 1]);
    }
  }
  return a[0] + a[1];
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
constexpr int kAdamTurn = 8 * kOptThreads;  // elements of a block per turn
constexpr int kAdamTurns = 2;               // turns of a chunk, fp32 states
constexpr int kAdamTurnsMx = 4;             // and 8-bit ones
template <bool MX>
constexpr int kAdamChunk = (MX ? kAdamTurnsMx : kAdamTurns) * kAdamTurn;
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
  float lr, b1, b2, omb1, omb2, k1, k2;  // omb = 1 - b; k1, k2: see adam_step
  uint32_t turn;                         // 0x9E3779B9 step
};

template <int CAP>
struct AdamTable {
  AdamEntry t[CAP];
  uint32_t end[CAP];
  int n;
  AdamHyper h;
  const float* clip;
};

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

// 32 bits for element i at this step: a multiply-and-shift mixer, so that neither neighbouring
// elements nor consecutive steps are correlated (with a plain multiple of the step averages drift
// by some percent).  The constants are published ones: the shifts 15, 12, 15 and their multipliers are
// a result of C. Wellons's search for 32-bit mixers of low bias ("Prospecting for Hash Functions",
// 2018), 0x85EBCA6B is a multiplier of A. Appleby's MurmurHash3, 0x9E3779B9 is 2^32 over the golden
// ratio.
__device__ __forceinline__ uint32_t dither_bits(uint32_t i, uint32_t turn) {
  uint32_t x = 0x85EBCA6Bu * i + turn;
  x = (x ^ (x >> 15)) * 0x2C1B3C6Du;
  x = (x ^ (x >> 12)) * 0x297A2D39u;
  return x ^ (x >> 15);
}

// Eight codes and their scale to fp32.
__device__ __forceinline__ Vec8 state_values(uint2 c, float scale) {
  Vec8 a;
  e4m3x4_to_f32(c.x, a.v);
  e4m3x4_to_f32(c.y, a.v + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) a.v[j] *= scale;
  return a;
}

// Four codes, the low bytes of c, in one word.
__device__ __forceinline__ uint32_t pack4(const uint32_t* c) {
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// Codes of eight values by dithered rounding to E4M3; all 32 lanes call this, four of them share a
// block of 32 elements.  V: the second moment.  x holds the values' dither bits.
// A value is rounded up when its place between two codes plus (r + 1/2) / 2^16 reaches 1.  With
// the value scaled to q (|q| <= 448) and by 2^-120 more, E4M3's exponents become fp32's lowest
// ones, its codes below 2^-6 fp32's subnormals, and the code is the upper bits of the sum of the
// fp32 pattern and 16 r + 8.  NaN and infinity give code 127 (NaN).
template <bool V>
__device__ __forceinline__ uint2 state_codes(const Vec8& a, const uint32_t (&x)[8], int* exponent) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, V ? a.v[j] : fabsf(a.v[j]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int s = mx_exponent(amax);
  *exponent = s;
  const float inv = __uint_as_float((uint32_t)(127 - s) << 23);
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t q = __float_as_uint(fabsf(a.v[j]) * inv * 0x1p-120f);
    c[j] = min((q + (((V ? x[j] << 4 : x[j] >> 12) & 0xFFFF0u) | 8u)) >> 20, 127u);
    if (V) c[j] = max(c[j], min(__float_as_uint(a.v[j]), 1u));  // v > 0 keeps a code
  }
  uint2 r = make_uint2(pack4(c), pack4(c + 4));
  if (!V) {  // the signs: the top bytes of the values
    uint32_t t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = __float_as_uint(a.v[j]);
    const uint32_t lo = __byte_perm(__byte_perm(t[0], t[1], 0x0073), __byte_perm(t[2], t[3], 0x0073), 0x5410);
    const uint32_t hi = __byte_perm(__byte_perm(t[4], t[5], 0x0073), __byte_perm(t[6], t[7], 0x0073), 0x5410);
    r.x |= lo & 0x80808080u;
    r.y |= hi & 0x80808080u;
  }
  return r;
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The step of eight elements in registers.  k1 = sqrt(c2) / c1 and k2 = eps / c1 carry the bias
// corrections c = 1 / (1 - beta^step).  FAST, for 8-bit states, whose kernel has two thirds of its
// issue slots taken: approximate root and reciprocal, together 2^-22 of the update lr m / root.  That
// is less than half a unit of w where |w| is 8 times the update or more, and up to 4 units where w is
// nothing but the update; the rounding of the states to codes moves the update by 2^-5 and more.
// With fp32 states every operation rounds once: 1416 -> 1417 us for 24 tensors of 14.7M weights, 53
// -> 54 for 96 small ones against the approximate forms.
template <bool FAST>
__device__ __forceinline__ void adam_step(const AdamHyper& h, float clip, float decay, const Vec8& g, Vec8& w, Vec8& m, Vec8& v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = g.v[j] * clip;
    m.v[j] = fmaf(h.b1, m.v[j], h.omb1 * gj);
    v.v[j] = fmaf(h.b2, v.v[j], h.omb2 * (gj * gj));
    const float update = FAST ? m.v[j] * rcp_approx(fmaf(sqrt_approx(v.v[j]), h.k1, h.k2))
                              : m.v[j] / fmaf(sqrtf(v.v[j]), h.k1, h.k2);
    w.v[j] = fmaf(-h.lr, fmaf(decay, w.v[j], update), w.v[j]);
  }
}

__device__ __forceinline__ uint2 load_codes(const void* p, int64_t i, int n) {
  if (n >= 8) return static_cast<const uint2*>(p)[i >> 3];
  uint2 c = make_uint2(0, 0);
  for (int j = 0; j < n; ++j) {
    const uint32_t b = static_cast<const uint8_t*>(p)[i + j];
    if (j < 4) c.x |= b << (8 * j);
    else c.y |= b << (8 * (j - 4));
  }
  return c;
}
__device__ __forceinline__ void store_codes(void* p, int64_t i, int n, uint2 c) {
  if (n >= 8) {
    static_cast<uint2*>(p)[i >> 3] = c;
  } else {
    for (int j = 0; j < n; ++j) static_cast<uint8_t*>(p)[i + j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

// A chunk whose end may be past the tensor's: eight elements per thread and turn.
template <bool P32, bool G32>
__device__ __forceinline__ void adam_chunk_f32(const AdamEntry& t, const AdamHyper& h, float clip, int64_t at) {
#pragma unroll 1
  for (int u = 0; u < kAdamTurns; ++u) {
    const int64_t i = at + u * kAdamTurn + 8 * threadIdx.x;
    const int n = (int)min((int64_t)8, t.numel - i);
    if (n <= 0) return;
    const Vec8 g = load8n<G32>(t.grad, i, n);
    Vec8 w = load8n<true>(P32 ? t.param : t.master, i, n);
    Vec8 m = load8n<true>(t.m, i, n), v = load8n<true>(t.v, i, n);
    adam_step<false>(h, clip, t.decay, g, w, m, v);
    store8n<true>(t.m, i, n, m);
    store8n<true>(t.v, i, n, v);
    store8n<true>(P32 ? t.param : t.master, i, n, w);
    if constexpr (!P32) store8n<false>(t.param, i, n, w);
  }
}

// What a thread reads for eight elements with 8-bit states.
template <bool G32>
struct AdamRaw {
  uint4 g[G32 ? 2 : 1];
  float4 w[2];
  uint2 m, v;
  uint32_t ms, vs;
};

// FULL: the whole chunk exists.  Then the next turn's data are loaded before this one's
// arithmetic (the kernel takes 68% of the issue slots at the copy rate).
template <bool P32, bool G32, bool FULL>
__device__ __forceinline__ void adam_chunk_mx(const AdamEntry& t, const AdamHyper& h, float clip, int64_t at) {
  void* const wp = P32 ? t.param : t.master;
  AdamRaw<G32> raw[2];
  auto load = [&](int u, AdamRaw<G32>& r) {
    const int64_t i = at + u * kAdamTurn + 8 * threadIdx.x;
    if constexpr (G32) {
      r.g[0] = static_cast<const uint4*>(t.grad)[i >> 2];
      r.g[1] = static_cast<const uint4*>(t.grad)[(i >> 2) + 1];
    } else {
      r.g[0] = static_cast<const uint4*>(t.grad)[i >> 3];
    }
    r.w[0] = static_cast<const float4*>(wp)[i >> 2];
    r.w[1] = static_cast<const float4*>(wp)[(i >> 2) + 1];
    r.m = static_cast<const uint2*>(t.m)[i >> 3];
    r.v = static_cast<const uint2*>(t.v)[i >> 3];
    r.ms = t.ms[i >> 5];
    r.vs = t.vs[i >> 5];
  };
  if constexpr (FULL) load(0, raw[0]);
#pragma unroll(FULL ? kAdamTurnsMx : 1)
  for (int u = 0; u < kAdamTurnsMx; ++u) {
    if (!FULL && at + u * kAdamTurn >= t.numel) break;
    const int64_t i = at + u * kAdamTurn + 8 * threadIdx.x;
    Vec8 g, w, m, v;
    int n = 8;
    if constexpr (FULL) {
      if (u + 1 < kAdamTurnsMx) load(u + 1, raw[(u + 1) & 1]);
      const AdamRaw<G32>& r = raw[u & 1];
      if constexpr (G32) {
        const uint4 a = r.g[0], b = r.g[1];
        g = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
             __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
      } else {
        g = unpack8(r.g[0]);
      }
      w = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
      m = state_values(r.m, e8m0(r.ms));
      v = state_values(r.v, e8m0(r.vs));
    } else {  // lanes past the end hold zeros and take part in the shuffles
      n = (int)min((int64_t)8, t.numel - i);
      g = load8n<G32>(t.grad, i, n);
      w = load8n<true>(wp, i, n);
      m = state_values(load_codes(t.m, i, n), n > 0 ? e8m0(t.ms[i >> 5]) : 0.0f);
      v = state_values(load_codes(t.v, i, n), n > 0 ? e8m0(t.vs[i >> 5]) : 0.0f);
    }
    adam_step<true>(h, clip, t.decay, g, w, m, v);
    uint32_t x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = dither_bits((uint32_t)i + j, h.turn);
    int ms, vs;
    const uint2 cm = state_codes<false>(m, x, &ms), cv = state_codes<true>(v, x, &vs);
    if (FULL) {
      store8<true>(wp, i >> 3, w);
      if constexpr (!P32) store8<false>(t.param, i >> 3, w);
      static_cast<uint2*>(t.m)[i >> 3] = cm;
      static_cast<uint2*>(t.v)[i >> 3] = cv;
    } else {
      store8n<true>(wp, i, n, w);
      if constexpr (!P32) store8n<false>(t.param, i, n, w);
      store_codes(t.m, i, n, cm);
      store_codes(t.v, i, n, cv);
    }
    if (n > 0 && (i & 31) == 0) {
      t.ms[i >> 5] = (uint8_t)(ms + 127);
      t.vs[i >> 5] = (uint8_t)(vs + 127);
    }
  }
}

template <bool MX, bool P32, bool G32>
__device__ __forceinline__ void adam_chunk(const AdamEntry& t, const AdamHyper& h, float clip, int64_t at) {
  if constexpr (!MX) adam_chunk_f32<P32, G32>(t, h, clip, at);
  else if (at + kAdamChunk<true> <= t.numel) adam_chunk_mx<P32, G32, true>(t, h, clip, at);
  else adam_chunk_mx<P32, G32, false>(t, h, clip, at);
}

// Bound by HBM: 28 bytes per bf16 weight with fp32 states, 16.1 with 8-bit ones.  Over 1.45e9
// weights (32 experts, d = 7168, F = 2048) it takes 5.79 ms (7.0 TB/s) with fp32 states and
// 3.46 ms (6.8 TB/s, the copy rate) with 8-bit ones.  For these, four blocks per SM at 64
// registers: with three (80 registers) 3.78 ms, two (123) 4.23, five (48, spilling) 4.54; chunks
// of 4096 elements (two turns, so less loaded ahead) 3.70 ms.
template <int CAP, bool MX>
__global__ void __launch_bounds__(kOptThreads, MX ? 4 : 1) adamw_kernel(const __grid_constant__ AdamTable<CAP> p) {
  const float clip = p.clip ? p.clip[1] : 1.0f;
  if (clip != clip) return;  // the gradients' norm is not finite: nothing changes
  const int k = tensor_of(p, blockIdx.x);
  const AdamEntry& t = p.t[k];
  const int64_t at = (int64_t)(blockIdx.x - (k ? p.end[k - 1] : 0u)) * kAdamChunk<MX>;
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
    c += chunks_of(t[j].numel, kAdamChunk<MX>);
    p.t[j] = AdamEntry{t[j].param, t[j].grad, t[j].master, t[j].exp_avg, t[j].exp_avg_sq, t[j].exp_avg_scale,
                       t[j].exp_avg_sq_scale, t[j].numel, (float)t[j].weight_decay, t[j].param_type == MOK_T_F32,
                       t[j].grad_type == MOK_T_F32};
    p.end[j] = (uint32_t)c;
  }
  if (c == 0) return cudaSuccess;
  if (c > 0x7fffffffLL) return cudaErrorInvalidValue;
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
  if (!is16(ws) || (reinterpret_cast<uintptr_t>(out) & 3u)) return MOK_ERR_UNSUPPORTED;
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
  if (reinterpret_cast<uintptr_t>(clip) & 3u) return MOK_ERR_UNSUPPORTED;
  const mok_adamw_args& a = *args;
  if (!(a.beta1 >= 0.0 && a.beta1 < 1.0) || !(a.beta2 >= 0.0 && a.beta2 < 1.0) || !(a.eps >= 1e-15) ||
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
  // m c1 / (sqrt(v c2) + eps) = m / (sqrt(v) k1 + k2)
  const double c1 = 1.0 / (1.0 - std::pow(a.beta1, (double)a.step)), c2 = 1.0 / (1.0 - std::pow(a.beta2, (double)a.step));
  h.k1 = (float)(std::sqrt(c2) / c1);
  h.k2 = (float)(a.eps / c1);
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
