// Balance loss, z loss, per-expert counts and the gradient of the router's logits.
//
// With c[s,e] the number of valid tokens of sequence s that chose expert e, n_s its valid tokens
// and n all of them, the balance loss is a sum over tokens once c is known:
//   balance = sum_t a_s <c_s, p_t>,  a_s = alpha E / (k n n_s),  s = the token's sequence,
//   dl_t = p_t (a_s (c_s - <c_s, p_t>) + b lse_t),  b = 2 z_coef / n,
// so one pass over the logits gives loss and gradient.  Counts are integer atomics (any order
// gives the same sums); the losses are summed per block and joined in a fixed order.
#include <algorithm>
#include <cmath>

#include "mok_vec.cuh"

namespace mok {

constexpr int kBalThreads = 256;
constexpr int kBalMaxBlocks = 2048;

struct BalanceParams {
  const float* logits;
  const int32_t* topk_idx;
  const int32_t* seq_offsets;  // [S + 1] or NULL
  const uint8_t* mask;         // or NULL
  const float* grad;           // or NULL
  int32_t* counts;             // [S, E]
  int32_t* n_seq;              // [S], then the total
  float2* partial;             // [blocks] {sum a <c, p>, sum lse^2}
  float* loss;
  float* dlogits;              // or NULL
  int* status;
  int64_t T;
  int S, E, k, blocks;
  float alpha, z_coef;
};

// Sequence of token t, or -1 when it is left out.
__device__ __forceinline__ int sequence_of(const BalanceParams& p, int64_t t) {
  if (p.mask && !p.mask[t]) return -1;
  if (!p.seq_offsets) return 0;
  int lo = 0, hi = p.S + 1;  // the first entry above t is in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.seq_offsets[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1 < p.S ? lo - 1 : -1;
}

__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(const __grid_constant__ BalanceParams p) {
  for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < p.T; t += (int64_t)gridDim.x * blockDim.x) {
    const int s = sequence_of(p, t);
    if (s < 0) continue;
    atomicAdd(p.n_seq + s, 1);
    atomicAdd(p.n_seq + p.S, 1);
    for (int j = 0; j < p.k; ++j) {
      const int e = p.topk_idx[t * p.k + j];
      if (e < 0 || e >= p.E) record_status(p.status, MOK_ERR_DEVICE_CHECK);
      else atomicAdd(p.counts + (int64_t)s * p.E + e, 1);
    }
  }
}

// One warp per token; lane i holds the 4-element vectors i, i + 32, ... of its logits.
__global__ void __launch_bounds__(kBalThreads) balance_grad_kernel(const __grid_constant__ BalanceParams p) {
  __shared__ float2 smem[kBalThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nvec = p.E / 4;
  const float n = (float)max(p.n_seq[p.S], 1);
  const float g = p.grad ? *p.grad : 1.0f;
  float sum_b = 0.0f, sum_z = 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * (kBalThreads / 32) + warp; t < p.T; t += (int64_t)gridDim.x * (kBalThreads / 32)) {
    const int s = sequence_of(p, t);
    float4 l[kMaxE / 128], c[kMaxE / 128];
    float top = -INFINITY;
    if (s >= 0) {
#pragma unroll
      for (int i = 0; i < kMaxE / 128; ++i) {
        const int v = lane + 32 * i;
        if (v < nvec) {
          l[i] = reinterpret_cast<const float4*>(p.logits)[t * nvec + v];
          const int4 ci = reinterpret_cast<const int4*>(p.counts)[(int64_t)s * nvec + v];
          c[i] = make_float4((float)ci.x, (float)ci.y, (float)ci.z, (float)ci.w);
        } else {
          l[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          c[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        top = fmaxf(top, fmaxf(fmaxf(l[i].x, l[i].y), fmaxf(l[i].z, l[i].w)));
      }
    }
    top = warp_max(top);
    const float base = top == -INFINITY ? 0.0f : top;
    float total = 0.0f, inner = 0.0f;
    if (s >= 0) {
#pragma unroll
      for (int i = 0; i < kMaxE / 128; ++i) {
        l[i] = make_float4(expf(l[i].x - base), expf(l[i].y - base), expf(l[i].z - base), expf(l[i].w - base));
        total += (l[i].x + l[i].y) + (l[i].z + l[i].w);
        inner = fmaf(c[i].x, l[i].x, fmaf(c[i].y, l[i].y, fmaf(c[i].z, l[i].z, fmaf(c[i].w, l[i].w, inner))));
      }
    }
    total = warp_sum(total);
    inner = warp_sum(inner);
    const bool live = s >= 0 && total != 0.0f;  // a NaN total stays live
    float a = 0.0f, b = 0.0f, inv = 0.0f;
    if (live) {
      inv = 1.0f / total;
      inner *= inv;
      a = p.alpha * (float)p.E / ((float)p.k * n * (float)p.n_seq[s]);
      const float lse = base + logf(total);
      b = 2.0f * p.z_coef / n * lse;
      sum_b += a * inner;
      sum_z += lse * lse;
    }
    if (p.dlogits) {
#pragma unroll
      for (int i = 0; i < kMaxE / 128; ++i) {
        const int v = lane + 32 * i;
        if (v < nvec) {
          float4 d = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (live) {
            const float q = g * inv;
            d = make_float4(l[i].x * q * (a * (c[i].x - inner) + b), l[i].y * q * (a * (c[i].y - inner) + b),
                            l[i].z * q * (a * (c[i].z - inner) + b), l[i].w * q * (a * (c[i].w - inner) + b));
          }
          reinterpret_cast<float4*>(p.dlogits)[t * nvec + v] = d;
        }
      }
    }
  }
  if (lane == 0) smem[warp] = make_float2(sum_b, sum_z);
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 a = make_float2(0.0f, 0.0f);
    for (int w = 0; w < kBalThreads / 32; ++w) {
      a.x += smem[w].x;
      a.y += smem[w].y;
    }
    p.partial[blockIdx.x] = a;
  }
}

__global__ void __launch_bounds__(32) balance_loss_kernel(const __grid_constant__ BalanceParams p) {
  double b = 0.0, z = 0.0;
  for (int i = threadIdx.x; i < p.blocks; i += 32) {
    b += p.partial[i].x;
    z += p.partial[i].y;
  }
  for (int o = 16; o; o >>= 1) {
    b += __shfl_xor_sync(0xffffffffu, b, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  if (threadIdx.x == 0) {
    p.loss[0] = (float)b;
    p.loss[1] = (float)(z * (double)p.z_coef / (double)max(p.n_seq[p.S], 1));
  }
}

static size_t balance_ws(int64_t S) {
  return 256 + (((size_t)S + 1) * sizeof(int32_t) + 255) / 256 * 256 + kBalMaxBlocks * sizeof(float2);
}

}  // namespace mok

extern "C" {

size_t mok_balance_loss_workspace_size(const mok_dims* dims, int64_t n_seqs) {
  using namespace mok;
  if (check_dims(dims) != MOK_OK || n_seqs < 1 || n_seqs > 0x7fffffffLL / dims->E) return 0;
  return balance_ws(n_seqs);
}

int mok_balance_loss(const mok_dims* dims, const float* logits, const int32_t* topk_idx,
                     const int32_t* seq_offsets, int64_t n_seqs, const uint8_t* token_mask,
                     float alpha, float z_coef, const float* grad, int32_t* counts, float* loss,
                     float* dlogits, void* ws, size_t ws_bytes, mok_stream_t stream) {
  using namespace mok;
  const int rc = check_dims(dims);
  if (rc != MOK_OK) return rc;
  if (n_seqs < 1 || (!seq_offsets && n_seqs != 1) || !std::isfinite(alpha) || !std::isfinite(z_coef))
    return MOK_ERR_INVALID_ARG;
  if (n_seqs > 0x7fffffffLL / dims->E) return MOK_ERR_UNSUPPORTED;
  if (!counts || !loss || !ws || (dims->T > 0 && (!logits || !topk_idx))) return MOK_ERR_INVALID_ARG;
  for (const void* q : {(const void*)logits, (const void*)counts, (const void*)dlogits, (const void*)ws})
    if (reinterpret_cast<uintptr_t>(q) & 15u) return MOK_ERR_UNSUPPORTED;
  if (ws_bytes < balance_ws(n_seqs)) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  BalanceParams p{};
  p.logits = logits;
  p.topk_idx = topk_idx;
  p.seq_offsets = seq_offsets;
  p.mask = token_mask;
  p.grad = grad;
  p.counts = counts;
  p.n_seq = reinterpret_cast<int32_t*>(w + 256);
  p.partial = reinterpret_cast<float2*>(w + balance_ws(n_seqs) - kBalMaxBlocks * sizeof(float2));
  p.loss = loss;
  p.dlogits = dlogits;
  p.status = static_cast<int*>(ws);
  p.T = dims->T;
  p.S = (int)n_seqs;
  p.E = dims->E;
  p.k = dims->k;
  p.alpha = alpha;
  p.z_coef = z_coef;
  const int64_t warps = kBalThreads / 32;
  p.blocks = (int)std::max<int64_t>(1, std::min<int64_t>((p.T + warps - 1) / warps, std::min(kBalMaxBlocks, num_sms() * 8)));
  cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * n_seqs * p.E, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(p.n_seq, 0, sizeof(int32_t) * (n_seqs + 1), s);
  if (e != cudaSuccess) return MOK_ERR_CUDA;
  prof_begin("balance_count", s);
  balance_count_kernel<<<(int)std::max<int64_t>(1, std::min<int64_t>((p.T + kBalThreads - 1) / kBalThreads, num_sms() * 8)), kBalThreads, 0, s>>>(p);
  prof_end(s);
  prof_begin("balance_grad", s);
  balance_grad_kernel<<<p.blocks, kBalThreads, 0, s>>>(p);
  prof_end(s);
  prof_begin("balance_loss", s);
  balance_loss_kernel<<<1, 32, 0, s>>>(p);
  prof_end(s);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(3);
  return MOK_OK;
}

}  // extern "C"
