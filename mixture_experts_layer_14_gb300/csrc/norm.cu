// RMS norm with the residual's addition and an optional MXFP8 output, and its backward pass.
//
//   h = x + residual,  rho = 1 / sqrt(mean(h^2) + eps),  v = h rho weight
//   ds = rho (g - xhat mean(g xhat)) + dres,  g = dy weight,  xhat = s rho;  dweight = sum dy xhat
//
// Each row is read once and kept in registers between its reduction and its outputs: thread i of
// the row's threads holds the 8-element vectors i, i + n, ..., so every access is a contiguous
// 512 bytes per warp and a 32-element MXFP8 block is held by four neighbouring lanes.
#include <algorithm>
#include <cmath>

#include "mok_mx.cuh"
#include "mok_vec.cuh"

namespace mok {

constexpr int kNormMaxD = 32768;

struct NormParams {
  const void* x;         // bf16
  const void* residual;  // or NULL
  const void* weight;
  void* y;               // bf16, or NULL
  void* residual_out;
  void* codes;           // or NULL
  uint8_t* scales;
  int64_t T, rows;       // rows: T, or T padded to 128 (scale atoms)
  int d;
  float eps;
  int weight_f32, atoms;
};

// Sum of two values over the row's threads (blockDim.x, a multiple of 32), the same in all of them.
__device__ __forceinline__ float2 row_sum(float a, float b, float2* smem) {
  a = warp_sum(a);
  b = warp_sum(b);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = make_float2(0.0f, 0.0f);
  for (int w = 0; w < warps; ++w) {
    t.x += smem[w].x;
    t.y += smem[w].y;
  }
  __syncthreads();
  return t;
}

__device__ __forceinline__ Vec8 load_weight(const void* w, int f32, int i) {
  return f32 ? load8<true>(w, i) : load8<false>(w, i);
}

// RES: 0 no residual, 1 bf16, 2 fp32.  V vectors per thread.
template <int V, int RES>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 smem[32];
  const int nvec = p.d >> 3;
  for (int64_t t = blockIdx.x; t < p.rows; t += gridDim.x) {
    if (t >= p.T) {  // padding rows of the scale atoms
      for (int kb = threadIdx.x; kb < p.d / 128; kb += blockDim.x)
        *reinterpret_cast<uint32_t*>(p.scales + sf_atom_word(t >> 7, kb, p.d / 128, (int)(t & 127))) = 0;
      continue;
    }
    Vec8 h[V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        h[i] = load8<false>(p.x, t * nvec + v);
        if constexpr (RES != 0) {
          const Vec8 r = load8<RES == 2>(p.residual, t * nvec + v);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i].v[j] += r.v[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i].v[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i].v[j], h[i].v[j], ss);
    }
    ss = row_sum(ss, 0.0f, smem).x;
    const float rho = 1.0f / sqrtf(ss / (float)p.d + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      const bool in = v < nvec;
      if (RES != 0 && in) store8<RES == 2>(p.residual_out, t * nvec + v, h[i]);
      if (in) {
        const Vec8 w = load_weight(p.weight, p.weight_f32, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i].v[j] = h[i].v[j] * rho * w.v[j];
        if (p.y) store8<false>(p.y, t * nvec + v, h[i]);
      }
      if (p.codes) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(h[i].v[j]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int s = mx_exponent(amax);
        const float inv = __uint_as_float((uint32_t)(127 - s) << 23);
        if (in) {
          uint2 q;
          q.x = e4m3x2(h[i].v[0] * inv, h[i].v[1] * inv) | (uint32_t)e4m3x2(h[i].v[2] * inv, h[i].v[3] * inv) << 16;
          q.y = e4m3x2(h[i].v[4] * inv, h[i].v[5] * inv) | (uint32_t)e4m3x2(h[i].v[6] * inv, h[i].v[7] * inv) << 16;
          static_cast<uint2*>(p.codes)[t * nvec + v] = q;
          if ((v & 3) == 0) {
            const int b = v >> 2;
            const int64_t at = p.atoms ? sf_atom_word(t >> 7, b >> 2, p.d / 128, (int)(t & 127)) + (b & 3)
                                       : t * (nvec >> 2) + b;
            p.scales[at] = (uint8_t)(s + 127);
          }
        }
      }
    }
  }
}

struct NormBwdParams {
  const void* dy;    // bf16
  const void* s;
  const void* dres;  // or NULL
  const void* weight;
  void* dx;          // bf16, or NULL
  void* dresidual;   // or NULL
  float* partial;    // [grid][d]
  int64_t T;
  int d;
  float eps;
  int weight_f32;
};

template <int V, bool F32>
__global__ void __launch_bounds__(1024) rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float2 smem[32];
  const int nvec = p.d >> 3;
  Vec8 dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i].v[j] = 0.0f;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    Vec8 s[V], dy[V];
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        s[i] = load8<F32>(p.s, t * nvec + v);
        dy[i] = load8<false>(p.dy, t * nvec + v);
        const Vec8 w = load_weight(p.weight, p.weight_f32, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(s[i].v[j], s[i].v[j], ss);
          dot = fmaf(s[i].v[j], dy[i].v[j] * w.v[j], dot);
        }
      }
    }
    const float2 sums = row_sum(ss, dot, smem);
    const float rho = 1.0f / sqrtf(sums.x / (float)p.d + p.eps);
    const float c = sums.y / (float)p.d * rho * rho;  // mean(g xhat) rho
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        const Vec8 w = load_weight(p.weight, p.weight_f32, v);
        Vec8 ds;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[i].v[j] = fmaf(dy[i].v[j], s[i].v[j] * rho, dw[i].v[j]);
          ds.v[j] = rho * (dy[i].v[j] * w.v[j] - s[i].v[j] * c);
        }
        if (p.dres) {
          const Vec8 r = load8<F32>(p.dres, t * nvec + v);
#pragma unroll
          for (int j = 0; j < 8; ++j) ds.v[j] += r.v[j];
        }
        if (p.dx) store8<false>(p.dx, t * nvec + v, ds);
        if (p.dresidual) store8<F32>(p.dresidual, t * nvec + v, ds);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nvec) store8<true>(p.partial + (int64_t)blockIdx.x * p.d, v, dw[i]);
  }
}

// dweight[c] = sum over the n partial rows, in order.
__global__ void __launch_bounds__(128) rms_norm_dweight_kernel(const float* __restrict__ partial, int n,
                                                               int d, float* __restrict__ dweight) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= d) return;
  float a = 0.0f;
  for (int r = 0; r < n; ++r) a += partial[(int64_t)r * d + c];
  dweight[c] = a;
}

static bool norm_sizes_ok(int64_t T, int d) {
  return T >= 0 && T <= 0x7fffffffLL / 8 && d > 0 && d <= kNormMaxD && d % 8 == 0;
}
// vectors per thread (1, 2 or 4) and threads of a row
static int norm_shape(int d, int* threads) {
  const int nvec = d / 8;
  const int v = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : 4;
  *threads = ((nvec + v - 1) / v + 31) / 32 * 32;
  return v;
}
static int norm_bwd_grid(int64_t T) { return (int)std::max<int64_t>(1, std::min<int64_t>(T, num_sms() * 2)); }
static bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace mok

extern "C" {

int mok_rms_norm(int64_t T, int d, float eps, const void* x, const void* residual, int res_type,
                 const void* weight, int weight_type, void* y, void* residual_out, void* codes,
                 void* scales, int scale_layout, mok_stream_t stream) {
  using namespace mok;
  if (!norm_sizes_ok(T, d)) return MOK_ERR_UNSUPPORTED;
  if (codes && d % 128) return MOK_ERR_UNSUPPORTED;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return MOK_ERR_INVALID_ARG;
  if ((res_type != MOK_T_BF16 && res_type != MOK_T_F32) || (weight_type != MOK_T_BF16 && weight_type != MOK_T_F32) ||
      (scale_layout != MOK_SCALES_ROWS && scale_layout != MOK_SCALES_ATOMS))
    return MOK_ERR_INVALID_ARG;
  if (T > 0 && (!x || !weight || (!y && !codes) || (codes && !scales))) return MOK_ERR_INVALID_ARG;
  if (T > 0 && (residual != nullptr) != (residual_out != nullptr)) return MOK_ERR_INVALID_ARG;
  for (const void* q : {x, residual, weight, (const void*)y, (const void*)residual_out, (const void*)codes, (const void*)scales})
    if (!is16(q)) return MOK_ERR_UNSUPPORTED;
  set_last_launches(0);
  if (T == 0) return MOK_OK;
  NormParams p{x, residual, weight, y, residual_out, codes, static_cast<uint8_t*>(scales), T, T, d, eps,
               weight_type == MOK_T_F32, scale_layout == MOK_SCALES_ATOMS};
  if (codes && p.atoms) p.rows = (T + 127) / 128 * 128;
  int threads;
  const int V = norm_shape(d, &threads);
  const int res = !residual ? 0 : res_type == MOK_T_F32 ? 2 : 1;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = (int)std::min<int64_t>(p.rows, 1 << 30);
  void (*k)(const NormParams) = nullptr;
  auto pick = [&](auto a, auto b, auto c) { k = res == 0 ? a : res == 1 ? b : c; };
  if (V == 1) pick(rms_norm_kernel<1, 0>, rms_norm_kernel<1, 1>, rms_norm_kernel<1, 2>);
  else if (V == 2) pick(rms_norm_kernel<2, 0>, rms_norm_kernel<2, 1>, rms_norm_kernel<2, 2>);
  else pick(rms_norm_kernel<4, 0>, rms_norm_kernel<4, 1>, rms_norm_kernel<4, 2>);
  prof_begin("rms_norm", s);
  k<<<grid, threads, 0, s>>>(p);
  prof_end(s);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(1);
  return MOK_OK;
}

size_t mok_rms_norm_workspace_size(int64_t T, int d) {
  using namespace mok;
  if (!norm_sizes_ok(T, d)) return 0;
  return 256 + sizeof(float) * (size_t)norm_bwd_grid(T) * d;
}

int mok_rms_norm_backward(int64_t T, int d, float eps, const void* dy, const void* s, int res_type,
                          const void* weight, int weight_type, const void* dres, void* dx,
                          void* dresidual, float* dweight, void* ws, size_t ws_bytes,
                          mok_stream_t stream) {
  using namespace mok;
  if (!norm_sizes_ok(T, d)) return MOK_ERR_UNSUPPORTED;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return MOK_ERR_INVALID_ARG;
  if ((res_type != MOK_T_BF16 && res_type != MOK_T_F32) || (weight_type != MOK_T_BF16 && weight_type != MOK_T_F32))
    return MOK_ERR_INVALID_ARG;
  if (!dweight || !ws || (T > 0 && (!dy || !s || !weight || (!dx && !dresidual)))) return MOK_ERR_INVALID_ARG;
  for (const void* q : {dy, s, weight, dres, (const void*)dx, (const void*)dresidual, (const void*)dweight, (const void*)ws})
    if (!is16(q)) return MOK_ERR_UNSUPPORTED;
  if (ws_bytes < mok_rms_norm_workspace_size(T, d)) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return cudaMemsetAsync(dweight, 0, sizeof(float) * d, st) == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
  float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  NormBwdParams p{dy, s, dres, weight, dx, dresidual, partial, T, d, eps, weight_type == MOK_T_F32};
  int threads;
  const int V = norm_shape(d, &threads);
  const int grid = norm_bwd_grid(T);
  const bool f = res_type == MOK_T_F32;
  auto k = V == 1 ? (f ? rms_norm_bwd_kernel<1, true> : rms_norm_bwd_kernel<1, false>)
         : V == 2 ? (f ? rms_norm_bwd_kernel<2, true> : rms_norm_bwd_kernel<2, false>)
                  : (f ? rms_norm_bwd_kernel<4, true> : rms_norm_bwd_kernel<4, false>);
  prof_begin("rms_norm_bwd", st);
  k<<<grid, threads, 0, st>>>(p);
  prof_end(st);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  prof_begin("rms_norm_dweight", st);
  rms_norm_dweight_kernel<<<(d + 127) / 128, 128, 0, st>>>(partial, grid, d, dweight);
  prof_end(st);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(2);
  return MOK_OK;
}

}  // extern "C"
